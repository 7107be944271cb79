"""One DP-SGD-RC step on a PyTorch model, with libdprc doing the work.

"Efficient DP-SGD for LLMs with Randomized Clipping" (papernotes.org,
"Method > Overall framework") lays the step out as:

  1. a forward pass that records, for every linear layer, its input
     activations A (B x T x d);
  2. a first backward pass that records the gradients G (B x T x p) with
     respect to each linear layer's output;
  3. per sample, per layer, the Hutchinson estimate of the squared norm of
     the weight gradient A_i^T G_i, summed over the layers;
  4. clip factors c_i = min(1, C / sqrt(n_i)) and a second backward pass of
     sum_i c_i L_i, which yields the clipped gradient sum sum_i c_i grad L_i;
  5. Gaussian noise sigma C N(0, I) added to that aggregated gradient.

`RandomizedClippingStep` does steps 2-5 around the caller's forward pass.
Steps 3-5 run in libdprc (Hutchinson: every layer and the clip factors of
the layer sum in one dprc_norm_hutch_layers_clip call; Hutch++: a
dprc_norm_hutchpp call per layer with accumulation, then dprc_clip_factors;
dprc_add_noise_at on each weight's gradient in place); PyTorch
provides the forward and backward passes and the memory.  The first backward
asks autograd only for the gradients with respect to the recorded layer
outputs, so no weight gradient is formed before the clip factors are known.

Scope: every trainable parameter must be the weight of an nn.Linear without
bias, the weight or bias of a `layers.Linear`, the weight or bias of a
`layers.LayerNorm`, or the weight of an embedding (`layers.Embedding`, or a plain
nn.Embedding); the norms of biases, embeddings and normalisations are exact and cheap
(dprc_embed_norm: a group sum of the output gradients; dprc_layernorm_grad: the
per-sample gradients, vectors of the width), other kinds would need their own per-sample
gradients, which the method does not cover.  Each layer runs once per
forward pass on inputs (B, ..., d) (every position between the batch and the
feature axis counts as a token), or on one sample after another; positions
that the samples share (an embedding of arange(T)) are expanded to [B, T] first.
A layer that runs twice and an input that mixes samples are refused, since a
sample's norm would not be that of its gradient.  The per-sample losses must not
couple samples.  The clipped gradient of an embedding or a normalisation is formed from the
recorded output gradients and the clip factors (dprc_embed_grad, dprc_layernorm_grad), so
the second backward stops at the linear parameters.  Projections are drawn fresh per
(layer, step) from a seeded
generator (a reading of the pages, which do not say how often P is redrawn):
P ~ N(0, 1/k) for Hutchinson, S and P ~ N(0, 1) for Hutch++.  Dividing the
noisy sum by the batch size is left to the optimiser.
"""

from __future__ import annotations

import torch

from . import binding as rnc
from . import layers as lay

_MIX = 0x9E3779B97F4A7C15
_BIAS_PLANS_KEPT = 16


def _seed(*parts):
    """A 63-bit seed from integers (splitmix-style mixing)."""
    h = 0
    for x in parts:
        h = (h ^ (int(x) & 0xFFFFFFFFFFFFFFFF)) * _MIX & 0xFFFFFFFFFFFFFFFF
        h ^= h >> 31
    return h & 0x7FFFFFFFFFFFFFFF


class RandomizedClippingStep:
    """DP-SGD-RC gradient step for the parameters of `model`.

    Args:
      model: the module; its trainable parameters must be those of bias-free
        nn.Linear, of `layers.Linear`, of `layers.LayerNorm` and of embeddings.
      C: clipping threshold.
      sigma: noise multiplier (0 disables the noise).
      k: projection width (Hutchinson) or r (Hutch++, k = 16).
      method: "hutch" or "hutchpp".
      seed: base seed of the projections and the noise.
    """

    def __init__(self, model, C, sigma, k=32, method="hutch", seed=0):
        if method not in ("hutch", "hutchpp"):
            raise ValueError("method must be 'hutch' or 'hutchpp'")
        self.model = model
        self.C = float(C)
        self.sigma = float(sigma)
        self.k = int(k)
        self.method = method
        self.seed = int(seed)
        self.layers = [m for m in model.modules()
                       if isinstance(m, (torch.nn.Linear, lay.Linear)) and m.weight.requires_grad]
        self.biased = [m for m in model.modules() if isinstance(m, lay.Linear)
                       and m.bias is not None and m.bias.requires_grad]
        self.embeddings = [m for m in model.modules()
                           if isinstance(m, (torch.nn.Embedding, lay.Embedding))
                           and m.weight.requires_grad]
        covered = {id(m.weight) for m in self.layers}
        for m in self.embeddings:
            if id(m.weight) in covered:
                raise ValueError("an embedding's weight is shared with another layer; the norm of "
                                 "a sum of two layers' gradients is not the sum of their norms")
            covered.add(id(m.weight))
            if getattr(m, "max_norm", None) is not None or getattr(m, "scale_grad_by_freq", False) \
                    or getattr(m, "sparse", False):
                raise ValueError("nn.Embedding with max_norm, scale_grad_by_freq or sparse "
                                 "gradients is not supported")
        covered |= {id(m.bias) for m in self.biased}
        self.norms = []
        for m in model.modules():
            own = [p for p in (m.weight, m.bias) if p is not None and p.requires_grad] \
                if isinstance(m, lay.LayerNorm) else []
            if not own:
                continue
            if any(id(p) in covered for p in own):
                raise ValueError("a normalisation's parameter is shared with another layer; the "
                                 "norm of a sum of two layers' gradients is not the sum of their "
                                 "norms")
            covered |= {id(p) for p in own}
            self.norms.append(m)
        for name, prm in model.named_parameters():
            if prm.requires_grad and id(prm) not in covered:
                raise ValueError(f"trainable parameter {name!r} has no per-sample norm here; covered "
                                 "are linear weights, the biases of layers.Linear, layers.LayerNorm and "
                                 "embeddings")
        for m in self.layers:
            if isinstance(m, torch.nn.Linear) and m.bias is not None and m.bias.requires_grad:
                raise ValueError("nn.Linear layers with a trainable bias are not supported")
        self._acts = {}
        self._outs = {}
        self._lasts = {}
        self._runs = {}
        self._mark = object()
        self._apart = set()
        recorded = self._recorded()
        self._handles = [m.register_forward_hook(self._record) for m in recorded]
        self._ws = {}
        self._bias_plans = {}

    def _recorded(self):
        return list(dict.fromkeys(self.layers + self.biased + self.embeddings + self.norms))

    def close(self):
        """Removes the hooks."""
        for h in self._handles:
            h.remove()
        self._handles = []

    def _record(self, module, inputs, output):
        # (a pass inside a backward pass is activation checkpointing's repetition
        # of one that is recorded)
        if torch.is_grad_enabled() and not lay._in_backward():
            self._acts[module] = inputs[0]
            self._outs[module] = output
            self._runs[module] = self._runs.get(module, 0) + 1
            if output.grad_fn is not None:
                output.grad_fn.metadata[self._mark] = module
            if isinstance(module, (lay.Linear, lay.LayerNorm)):
                self._lasts[module] = module._last

    def _refuse_repeats(self, losses):
        """Raises if a layer stands in the losses' graph more than once."""
        if all(n == 1 for n in self._runs.values()):
            return
        # (several passes may have been made and only the last one be stepped on)
        todo, seen, met = [losses.grad_fn], set(), set()
        while todo:
            node = todo.pop()
            if node is None or node in seen:
                continue
            seen.add(node)
            m = node.metadata.get(self._mark)
            if m is not None and m in met:
                raise ValueError(f"{type(m).__name__} runs more than once in the losses' forward "
                                 "pass; its gradient is a sum whose norm is not covered")
            met.add(m)
            todo.extend(n for n, _ in node.next_functions)

    def _refuse_mixed(self, recorded, losses):
        """Raises unless every layer's positions fall into B equal shares, one after
        another, that belong to one sample each.  Inputs with the batch and a
        position axis in front are taken at their word.  Others (rows, packed
        sequences, an embedding's [B]) may be shared positions as well: once per layer and
        share, the first and the last sample's losses must have no gradient
        outside their own share."""
        B = losses.shape[0]
        shares = {}
        for m in recorded if B > 1 else ():
            x = self._acts[m]
            table = m in self.embeddings
            positions = x.numel() if table else x.numel() // max(x.shape[-1], 1)
            if positions % B != 0:
                raise ValueError(f"{type(m).__name__}: an input of shape {tuple(x.shape)} does not "
                                 f"hold the positions of {B} samples; shared positions need an "
                                 "entry for every sample")
            whole = x.dim() > 1 and x.shape[0] == B  # (an embedding's [B] has one axis)
            if not whole and (m, positions // B) not in self._apart:
                shares[m] = positions // B
        for i in (0, B - 1) if shares else ():
            grads = torch.autograd.grad(losses[i], [self._outs[m] for m in shares],
                                        retain_graph=True, allow_unused=True)
            for (m, n), g in zip(shares.items(), grads):
                if g is None:
                    continue
                g = g.reshape(B * n, -1)
                # (a NaN is what 0 becomes beside an infinity)
                if any(bool(((r != 0) & (r == r)).any()) for r in (g[:i * n], g[(i + 1) * n:])):
                    raise ValueError(f"{type(m).__name__}: positions of an input of shape "
                                     f"{tuple(self._acts[m].shape)} belong to more than one sample")
        self._apart.update(shares.items())

    def parameters(self):
        """The trainable parameters in the order the noise stream runs over
        them: linear weights, biases, embeddings, normalisations."""
        return ([m.weight for m in self.layers] + [m.bias for m in self.biased]
                + [m.weight for m in self.embeddings]
                + [p for m in self.norms for p in self._norm_parameters(m)])

    @staticmethod
    def _norm_parameters(m):
        return [p for p in (m.weight, m.bias) if p is not None and p.requires_grad]

    def _norm_grad(self, m, G, n=None, c=None):
        """A normalisation's per-sample norms into n, or with the clip factors c its clipped
        gradient into its parameters."""
        X = lay._dense(self._acts[m]).reshape(G.shape)
        stats = self._lasts[m].reshape(*G.shape[:-1], 2)
        w = None if m.weight is None else lay._dense(m.weight)
        gain = m.weight is not None and m.weight.requires_grad
        shift = m.bias is not None and m.bias.requires_grad
        if n is not None and gain:
            rnc.dprc_layernorm_grad(G, X, stats, w, center=m.center, n=n, norm_of_bias=shift,
                                    accumulate=True)
        elif n is not None:
            rnc.dprc_embed_norm(G, self._bias_plan(G.shape[0], G.shape[1], G.device), n,
                                accumulate=True)
        else:
            dW = torch.empty_like(m.weight) if gain else None
            db = torch.empty_like(m.bias) if shift else None
            rnc.dprc_layernorm_grad(G, X, stats, w, center=m.center, dW=dW, db=db, c=c)
            if gain:
                m.weight.grad = dW
            if shift:
                m.bias.grad = db

    def _bias_plan(self, B, T, device):
        """The plan of the one-row embedding that a bias is: every position 0.  Kept
        for the last sizes; the current stream waits for the one that made it."""
        def make():
            return rnc.dprc_embed_plan(torch.zeros((B, T), dtype=torch.int32, device=device), 1)

        on_gpu = device.type == "cuda"
        if on_gpu and torch.cuda.is_current_stream_capturing():
            return make()  # a graph cannot wait for what was recorded outside of it
        key = (B, T, device)
        if key not in self._bias_plans:
            plan, made = make(), None
            if on_gpu:
                made = torch.cuda.Event()
                made.record(torch.cuda.current_stream(device))
            if len(self._bias_plans) == _BIAS_PLANS_KEPT:
                del self._bias_plans[next(iter(self._bias_plans))]
            self._bias_plans[key] = plan, made
        plan, made = self._bias_plans[key]
        if on_gpu:
            stream = torch.cuda.current_stream(device)
            stream.wait_event(made)
            plan.buf.record_stream(stream)
        return plan

    def projections(self, step):
        """The projection(s) of every layer for `step`: P [p][k] (Hutchinson)
        or (S, P) [p][k] (Hutch++), in the layer's dtype, on its device."""
        out = []
        for j, m in enumerate(self.layers):
            p = m.out_features
            dev, dt = m.weight.device, m.weight.dtype
            g = torch.Generator(device=dev)
            g.manual_seed(_seed(self.seed, 1, j, step))
            if self.method == "hutch":
                P = (torch.randn(p, self.k, generator=g, device=dev) / self.k ** 0.5).to(dt)
                out.append(P)
            else:
                S = torch.randn(p, self.k, generator=g, device=dev).to(dt)
                P = torch.randn(p, self.k, generator=g, device=dev).to(dt)
                out.append((S, P))
        return out

    def _layers_workspace(self, As, Gs, proj):
        B, T = As[0].shape[0], As[0].shape[1]
        k = max(P.shape[1] for P in proj)
        need = rnc.dprc_workspace_bytes(rnc.DPRC_OP_HUTCH_LAYERS, rnc._dtype_code(As[0]), B, T,
                                        max(A.shape[2] for A in As), max(G.shape[2] for G in Gs),
                                        k)
        key = (As[0].device, rnc.DPRC_OP_HUTCH_LAYERS)
        ws = self._ws.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.zeros(need, dtype=torch.uint8, device=As[0].device)  # zeroed once
            self._ws[key] = ws
        return ws

    def _workspace(self, op, A, B, T, d, p, k):
        need = rnc.dprc_workspace_bytes(op, rnc._dtype_code(A), B, T, d, p, k)
        key = (A.device, op)
        ws = self._ws.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.zeros(need, dtype=torch.uint8, device=A.device)  # zeroed once
            self._ws[key] = ws
        return ws

    def __call__(self, per_sample_losses, step, projections=None):
        """Runs steps 2-5 for losses L_i = per_sample_losses [B] of the forward
        pass just made.  Leaves sum_i c_i grad L_i (+ noise) in the weights'
        .grad and returns {"n": n, "c": c} (fp32 [B] on the device)."""
        losses = per_sample_losses
        if losses.dim() != 1:
            raise ValueError("per_sample_losses must have shape [B]")
        B = losses.shape[0]
        recorded = self._recorded()
        if any(m not in self._outs for m in self.layers):
            raise RuntimeError("no forward pass recorded for some linear layers")
        if any(m not in self._outs for m in recorded):
            raise RuntimeError("no forward pass recorded for some layers")
        self._refuse_repeats(losses)
        # step 2: gradients with respect to the layer outputs only
        fused = [m for m in recorded if isinstance(m, (lay.Linear, lay.LayerNorm))]
        for m in fused:
            m.norm_pass = True
        try:
            self._refuse_mixed(recorded, losses)
            grads = torch.autograd.grad(losses.sum(), [self._outs[m] for m in recorded],
                                        retain_graph=True)
        finally:
            for m in fused:
                m.norm_pass = False
        G_of = {}
        for m, G in zip(recorded, grads):
            dt = m.weight.dtype if m in self.embeddings else self._acts[m].dtype
            G = lay._dense(G.to(dt))
            if isinstance(m, lay.Linear):
                G = m.preactivation_grad(G, self._lasts[m])
            G_of[m] = G.reshape(B, -1, G.shape[-1])
        proj = self.projections(step) if projections is None else projections
        # step 3: layerwise sum of the per-sample estimates
        n = torch.zeros(B, dtype=torch.float32, device=losses.device)
        c = torch.empty_like(n)
        # the exact norms of biases and embeddings come first, the estimates add
        for m in self.biased:
            G = G_of[m]
            rnc.dprc_embed_norm(G, self._bias_plan(B, G.shape[1], G.device), n, accumulate=True)
        for m in self.norms:
            self._norm_grad(m, G_of[m], n=n)
        plans = {}
        for m in self.embeddings:
            tokens = self._acts[m].detach().reshape(B, -1)
            if getattr(m, "padding_idx", None) is not None:
                tokens = torch.where(tokens == m.padding_idx, -1, tokens)
            plans[m] = rnc.dprc_embed_plan(lay._dense(tokens), m.weight.shape[0])
            rnc.dprc_embed_norm(G_of[m], plans[m], n, scale=getattr(m, "scale", 1.0),
                                accumulate=True)
        As, Gs = [], []
        for m in self.layers:
            A = self._acts[m]
            # (B, ..., d): every position between batch and features is a token
            As.append(A.detach().reshape(B, -1, A.shape[-1]).contiguous())
            Gs.append(G_of[m])
        more = bool(self.biased or self.embeddings or self.norms)
        one_call = (self.method == "hutch" and As and len({A.shape[1] for A in As}) == 1
                    and len({P.shape[1] for P in proj}) == 1 and len({A.dtype for A in As}) == 1)
        if one_call:
            # every layer in one call (persistent launches of up to 56 layers),
            # the clip factors of the layer sum in the same call (step 4)
            ws = self._layers_workspace(As, Gs, proj)
            rnc.dprc_norm_hutch_layers(As, Gs, proj, n, accumulate=more, ws=ws, C=self.C, c=c)
        else:
            last = len(self.layers) - 1
            for j, (A, G) in enumerate(zip(As, Gs)):
                Bt, T, d = A.shape
                p = G.shape[-1]
                if self.method == "hutch":
                    ws = self._workspace(rnc.DPRC_OP_HUTCH, A, Bt, T, d, p, proj[j].shape[1])
                    if j == last:  # step 4's clip factors come with the last layer's norms
                        rnc.dprc_norm_hutch_clip(A, G, proj[j], n, self.C, c,
                                                 accumulate=more or j > 0, ws=ws)
                    else:
                        rnc.dprc_norm_hutch(A, G, proj[j], n, accumulate=more or j > 0, ws=ws)
                else:
                    S, P = proj[j]
                    ws = self._workspace(rnc.DPRC_OP_HUTCHPP, A, Bt, T, d, p, S.shape[1])
                    rnc.dprc_norm_hutchpp(A, G, S, P, n, accumulate=more or j > 0, ws=ws)
        # step 4: clip factors (Hutch++: here) and the rescaled second backward
        if self.method != "hutch" or not As:
            rnc.dprc_clip_factors(n, self.C, c)
        for prm in self.parameters():
            prm.grad = None
        loss = (c.to(losses.dtype) * losses).sum()
        if not more:
            loss.backward()
        elif self.layers or self.biased:
            torch.autograd.backward(loss, inputs=[m.weight for m in self.layers]
                                    + [m.bias for m in self.biased])
        for m in self.embeddings:
            dW = torch.empty_like(m.weight)
            rnc.dprc_embed_grad(G_of[m], plans[m], dW, c=c, scale=getattr(m, "scale", 1.0))
            m.weight.grad = dW
        for m in self.norms:
            self._norm_grad(m, G_of[m], c=c)
        # step 5: noise on the aggregated gradient, in place: the parameters'
        # gradients laid end to end in parameters() order are that gradient, and each
        # gets the stretch of the one noise stream its position there selects
        if self.sigma > 0.0:
            off = 0
            for prm in self.parameters():
                g = prm.grad
                if not g.is_contiguous():
                    raise RuntimeError("weight gradients must be contiguous")
                rnc.dprc_add_noise_at(g, off, self.sigma, self.C, _seed(self.seed, 2), step)
                off += g.numel()
        self._acts.clear()
        self._outs.clear()
        self._lasts.clear()
        self._runs.clear()
        for m in recorded:
            if isinstance(m, (lay.Linear, lay.LayerNorm)):
                m._last = None
        return {"n": n, "c": c}
