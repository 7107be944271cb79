"""The clipping step's kept data on another stream than the one it was made on."""

import numpy as np
import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from oracle import operators as ops
from randomized_norm_clipping_gb300 import layers as lay
from randomized_norm_clipping_gb300.step import RandomizedClippingStep
from randomized_norm_clipping_gb300.workloads import to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_a_bias_plan_waits_for_the_stream_that_makes_it():
    model = lay.Linear(8, 8, bias=True).to(DEV)
    step = RandomizedClippingStep(model, C=1.0, sigma=0.0)
    G = torch.randint(-2, 3, (3, 500, 8), device=DEV).float()
    n = torch.zeros(3, device=DEV)
    made, used = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(made):
        torch.cuda._sleep(200_000_000)  # some 0.1 s of work ahead of it
        step._bias_plan(3, 500, G.device)
    with torch.cuda.stream(used):
        rnc.dprc_embed_norm(G, step._bias_plan(3, 500, G.device), n)
    used.synchronize()
    tok = np.zeros((3, 500), dtype=np.int64)
    assert np.array_equal(to_f64(n), ops.embed_norm(to_f64(G), tok, 1))
    torch.cuda.synchronize()
    step.close()
