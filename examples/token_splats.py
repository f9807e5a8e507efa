"""A small network that predicts Gaussians, trained through the rasterizer.

Every token becomes one Gaussian.  The tokens of all scenes stand in one
ragged batch, a document per scene; a layer mixes them with the token
operators (norm and rotary position of queries and keys, attention within the
document, gated scan along it) and a last product writes the Gaussians' planes.
Each scene is rendered against its image, and the gradients the rasterizer
returns for its Gaussians go back through the network.  ``step`` is the same
layer in serving: one new token for every document, with the keys and values
cached and the scan's state carried on.  ``Served`` is the layer as it is served in
8 bits: its products' weights and its cache are kept in 8 (the cache also in 4)
bits, and a prompt that all requests share is in the cache once.

    python examples/token_splats.py [steps]      trains a layer

A program that serves makes a ``Served`` of the trained layer, gives it the prompt
with ``take_prompt`` and asks it for a token of every request with ``step``.

In training the matrix products are torch's; everything else on the tokens is the
library's, in serving in 8 bits its products too.
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from differentiable_rasterization_amd import raster, scenes  # noqa: E402

HALF = torch.bfloat16
Y00 = scenes.Y00


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _space(size):
    return torch.empty((max(size, 256),), dtype=torch.uint8, device="cuda")


class TokenLayer:
    """qkv product, norm + rotary, attention, gated scan, Gaussian head."""
    OUT = 14  # mean 3, log-scale 3, quaternion 4, opacity logit 1, colour 3

    def __init__(self, channels=128, heads_q=4, heads_k=2, dim=32, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda i, o, s=1.0: torch.randn((i, o), generator=gen, device="cuda") * s / i ** 0.5
        self.C, self.hq, self.hk, self.D = channels, heads_q, heads_k, dim
        self.w = {"qkv": w(channels, (heads_q + 2 * heads_k) * dim),
                  "out": w(heads_q * dim, channels), "gate": w(channels, 2 * channels),
                  "head": w(channels, self.OUT, 0.1),
                  "wq": torch.ones(dim, device="cuda"), "wk": torch.ones(dim, device="cuda")}
        self.inv_freq = (1000.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))).float()
        self.qk = raster.qk_config(HALF, heads_q, heads_k, dim)
        self.attention = raster.attention_config(HALF, heads_q, heads_k, dim, dim ** -0.5,
                                                 causal=True, softcap=20.0)
        self.scan = raster.scan_config(HALF, channels, coupled=True)

    def _project(self, x):
        qkv = (x @ self.w["qkv"].to(HALF)).view(len(x), self.hq + 2 * self.hk, self.D)
        return qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hk], qkv[:, self.hq + self.hk:]

    def _turn(self, positions, q, k):
        q2, k2 = torch.empty_like(q), torch.empty_like(k)
        raster.gs_qk_norm_rope_fwd(self.qk, len(q), positions, self.inv_freq, self.w["wq"],
                                   self.w["wk"], q, k, q2, k2)
        return q2, k2

    def forward(self, x, positions, docs):
        """x [tokens, C] (bfloat16) to the head's outputs [tokens, 14] (fp32);
        keeps what backward needs."""
        n = len(x)
        q, k, v = self._project(x)
        q2, k2 = self._turn(positions, q, k)
        o = torch.empty_like(q2)
        lse = torch.empty((self.hq, n), device="cuda")
        size = raster.gs_attention_fwd_workspace_size(self.attention, docs, n, n)
        raster.gs_attention_fwd(self.attention, docs, n, n, q2, k2, v, o, lse, _space(size), size)
        y = x + o.view(n, -1) @ self.w["out"].to(HALF)
        gx = y @ self.w["gate"].to(HALF)
        h = torch.empty_like(x)
        saved = _space(raster.gs_gated_scan_saved_size(self.scan, docs, n))
        size = raster.gs_gated_scan_fwd_workspace_size(self.scan, docs, n)
        raster.gs_gated_scan_fwd(self.scan, docs, n, gx[:, :self.C], gx[:, self.C:], None, h, None,
                                 saved, _space(size), size)
        z = (y + h).float()
        self.kept = (x, positions, docs, q, k, v, q2, k2, o, lse, y, gx, saved, z)
        return z @ self.w["head"]

    def backward(self, dp):
        """Gradients of the weights from those of the head's outputs."""
        x, positions, docs, q, k, v, q2, k2, o, lse, y, gx, saved, z = self.kept
        n, g = len(x), {}
        g["head"] = z.T @ dp
        dz = (dp @ self.w["head"].T).to(HALF)
        dgx = torch.empty_like(gx)
        size = raster.gs_gated_scan_bwd_workspace_size(self.scan, docs, n)
        raster.gs_gated_scan_bwd(self.scan, docs, n, gx[:, :self.C], gx[:, self.C:], saved, dz,
                                 None, dgx[:, :self.C], dgx[:, self.C:], None, _space(size), size)
        g["gate"] = (y.T @ dgx).float()
        dy = dz + dgx @ self.w["gate"].to(HALF).T
        g["out"] = (o.view(n, -1).T @ dy).float()
        do = (dy @ self.w["out"].to(HALF).T).view_as(o)
        dq2, dk2 = torch.empty_like(q2), torch.empty_like(k2)
        dqkv = torch.empty((n, self.hq + 2 * self.hk, self.D), dtype=HALF, device="cuda")
        dq, dk = dqkv[:, :self.hq], dqkv[:, self.hq:self.hq + self.hk]
        size = raster.gs_attention_bwd_workspace_size(self.attention, docs, n, n)
        raster.gs_attention_bwd(self.attention, docs, n, n, q2, k2, v, o, lse, do, dq2, dk2,
                                dqkv[:, self.hq + self.hk:], _space(size), size)
        g["wq"], g["wk"] = torch.empty_like(self.w["wq"]), torch.empty_like(self.w["wk"])
        size = raster.gs_qk_norm_rope_bwd_workspace_size(self.qk, n)
        raster.gs_qk_norm_rope_bwd(self.qk, n, positions, self.inv_freq, self.w["wq"],
                                   self.w["wk"], q, k, dq2, dk2, dq, dk, g["wq"], g["wk"],
                                   _space(size), size)
        g["qkv"] = (x.T @ dqkv.view(n, -1)).float()
        return g

    def start(self, requests, room):
        """A cache with room for so many tokens of every request."""
        z = lambda *shape: torch.zeros(shape, dtype=HALF, device="cuda")
        return {"k": z(requests * room, self.hk, self.D), "v": z(requests * room, self.hk, self.D),
                "state": torch.zeros((requests, self.C), device="cuda"), "room": room, "used": 0,
                "rows": torch.arange(requests, device="cuda") * room}

    def step(self, cache, x):
        """One new token of every request, x [requests, C]."""
        n, at = len(x), cache["used"]
        assert at < cache["room"]
        q, k, v = self._project(x)
        q2, k2 = self._turn(torch.full((n,), at, dtype=torch.int32, device="cuda"), q, k)
        cache["k"][cache["rows"] + at], cache["v"][cache["rows"] + at] = k2, v
        cache["used"] = at + 1
        one = torch.ones(n, dtype=torch.int32, device="cuda")
        docs = raster.documents(torch.arange(n, dtype=torch.int32, device="cuda"), one,
                                cache["rows"].int(), one * (at + 1), max_q_len=1,
                                max_k_len=at + 1)
        o = torch.empty_like(q2)
        rows = cache["k"].shape[0]
        size = raster.gs_attention_fwd_workspace_size(self.attention, docs, n, rows)
        raster.gs_attention_fwd(self.attention, docs, n, rows, q2, cache["k"], cache["v"], o, None,
                                _space(size), size)
        y = x + o.view(n, -1) @ self.w["out"].to(HALF)
        gx = y @ self.w["gate"].to(HALF)
        h = torch.empty_like(x)
        raster.gs_gated_scan_fwd(self.scan, docs, n, gx[:, :self.C], gx[:, self.C:],
                                 cache["state"], h, cache["state"], None, None, 0)
        return (y + h).float() @ self.w["head"]


class Served:
    """A trained layer with 8-bit weights, for requests that share a prompt."""

    def __init__(self, layer, requests, room, prompt=0, bits=8):
        self.layer, self.bits, self.requests, self.room = layer, bits, requests, room
        self.prompt, self.used, self.rows = prompt, 0, prompt + requests * room
        self.w = {}
        for name in ("qkv", "out", "gate"):
            w = layer.w[name].T.contiguous()                     # [outputs, inputs]
            codes = torch.empty(w.shape, dtype=torch.int8, device="cuda")
            scales = torch.empty(len(w), device="cuda")
            raster.gs_quantize_rows(w.dtype, *w.shape, w, codes, scales)
            self.w[name] = codes, scales
        self.cfg = raster.cache_config(HALF, layer.hk, layer.D)
        size = (self.rows, layer.hk, layer.D * bits // 8)
        self.cache = [raster.codes(torch.zeros(size, dtype=torch.uint8, device="cuda"),
                                   *torch.zeros((2, layer.hk, self.rows), device="cuda"), bits)
                      for _ in "kv"]
        self.state = torch.zeros((requests, layer.C), device="cuda")

    def _product(self, name, x):
        codes, scales = self.w[name]
        cfg = raster.linear_config(HALF, codes.shape[1], codes.shape[0])
        y = torch.empty((len(x), codes.shape[0]), dtype=HALF, device="cuda")
        size = raster.gs_linear_i8_workspace_size(cfg, len(x))
        raster.gs_linear_i8(cfg, len(x), x, codes, scales, None, y, _space(size), size)
        return y

    def _run(self, x, positions, docs, shared, state):
        """New tokens of all documents: into the cache, and through the layer."""
        layer, n = self.layer, len(x)
        qkv = self._product("qkv", x).view(n, layer.hq + 2 * layer.hk, layer.D)
        q, k = qkv[:, :layer.hq], qkv[:, layer.hq:layer.hq + layer.hk]
        q2, k2 = layer._turn(positions, q, k)
        raster.gs_cache_write(self.cfg, docs, n, self.rows, k2, qkv[:, layer.hq + layer.hk:],
                              *self.cache)
        o = torch.empty_like(q2)
        size = raster.gs_cached_attention_fwd_workspace_size(layer.attention, self.bits, docs,
                                                             shared, n, self.rows)
        raster.gs_cached_attention_fwd(layer.attention, docs, shared, n, self.rows, q2,
                                       *self.cache, o, None, _space(size), size)
        y = x + self._product("out", o.view(n, -1))
        gx = self._product("gate", y)
        h = torch.empty_like(x)
        size = raster.gs_gated_scan_fwd_workspace_size(layer.scan, docs, n)
        raster.gs_gated_scan_fwd(layer.scan, docs, n, gx[:, :layer.C], gx[:, layer.C:], state, h,
                                 state, None, _space(size), size)
        return (y + h).float() @ layer.w["head"]

    def take_prompt(self, x):
        """The shared prompt, x [prompt, C]: its keys stand in front of all requests."""
        n = len(x)
        assert n == self.prompt and self.used == 0
        docs = raster.documents(_ints([0]), _ints([n]), _ints([0]), _ints([n]), max_q_len=n,
                                max_k_len=n)
        state = torch.zeros((1, self.layer.C), device="cuda")
        p = self._run(x, torch.arange(n, dtype=torch.int32, device="cuda"), docs, None, state)
        self.state.copy_(state.expand_as(self.state))
        return p

    def step(self, x):
        """One new token of every request, x [requests, C]."""
        n, at = len(x), self.used
        assert n == self.requests and at < self.room
        one = torch.ones(n, dtype=torch.int32, device="cuda")
        first = torch.arange(n, dtype=torch.int32, device="cuda")
        docs = raster.documents(first, one, self.prompt + first * self.room, one * (at + 1),
                                max_q_len=1, max_k_len=at + 1)
        shared = None
        if self.prompt:
            shared = raster.documents(_ints([0]), _ints([n]), _ints([0]), _ints([self.prompt]),
                                      max_q_len=n, max_k_len=self.prompt)
        self.used = at + 1
        return self._run(x, one * (self.prompt + at), docs, shared, self.state)


class Adam:
    def __init__(self, weights, rate):
        self.w, self.rate, self.t = weights, rate, 0
        self.m = {n: torch.zeros_like(t) for n, t in weights.items()}
        self.v = {n: torch.zeros_like(t) for n, t in weights.items()}

    def step(self, grads):
        self.t += 1
        for n, g in grads.items():
            self.m[n].mul_(0.9).add_(g, alpha=0.1)
            self.v[n].mul_(0.99).addcmul_(g, g, value=0.01)
            m, v = self.m[n] / (1 - 0.9 ** self.t), self.v[n] / (1 - 0.99 ** self.t)
            self.w[n].sub_(self.rate * m / (v.sqrt() + 1e-8))


class Scenes:
    """Scenes of different sizes: their images, and per Gaussian what the
    network starts from (its base values, which the head's outputs move)."""

    def __init__(self, sizes, seed=1):
        self.sizes, self.starts = sizes, np.cumsum([0] + sizes[:-1]).tolist()
        self.cam, self.frames, self.targets, base = None, [], [], []
        for i, n in enumerate(sizes):
            scene, cam = scenes.tiny_scene(n=n, seed=seed + i)
            self.cam = cam
            truth = raster.Gaussians.from_scene(scene)
            frame = raster.Frame(n, 0, cam.width, cam.height)
            frame.forward(truth, cam)
            self.targets.append(frame.image.clone())
            self.frames.append(frame)
            gen = torch.Generator(device="cuda").manual_seed(seed + 100 + i)
            noise = lambda p: torch.randn((p, n), generator=gen, device="cuda")
            o = truth.opacities.clamp(0.02, 0.98)
            base.append(torch.cat((truth.means + 0.05 * noise(3), truth.scales.log() +
                                   0.2 * noise(3), truth.quats, torch.log(o / (1 - o)),
                                   truth.sh + 0.5 * noise(3))))
        self.base = torch.cat(base, 1)                           # [14, tokens]
        self.docs = raster.documents(_ints(self.starts), _ints(sizes), max_q_len=max(sizes))
        self.positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in sizes]).cuda()

    def tokens(self, channels, seed=7):
        """Input features: the base values and fixed random features of them."""
        gen = torch.Generator(device="cuda").manual_seed(seed)
        w = torch.randn((self.base.shape[0], channels), generator=gen, device="cuda")
        return torch.tanh(0.5 * self.base.T @ w).to(HALF)

    def loss(self, p):
        """Sum of squared differences over all scenes' pixels, and its gradient
        with respect to p [tokens, 14]."""
        raw = self.base + p.T
        total, dp = 0.0, torch.zeros_like(raw)
        for s, n, frame, target in zip(self.starts, self.sizes, self.frames, self.targets):
            r = raw[:, s:s + n].contiguous()
            g = raster.Gaussians(r[0:3].contiguous(), r[3:6].exp(), r[6:10].contiguous(),
                                 torch.sigmoid(r[10:11]), r[11:14].contiguous(), 0, n)
            frame.forward(g, self.cam)
            frame.loss_grad(target, 0)
            frame.backward(g)
            total += float(frame.loss)
            d = dp[:, s:s + n]
            d[0:3], d[3:6] = frame.g_means, frame.g_scales * g.scales
            d[6:10], d[11:14] = frame.g_quats, frame.g_sh
            d[10] = frame.g_opacities * (g.opacities * (1 - g.opacities))[0]
        return total, dp.T.contiguous()


def train(steps=60, sizes=(300, 97, 512, 33), rate=5e-4, report=None):
    """Losses of the training steps, and the layer."""
    data = Scenes(list(sizes))
    layer = TokenLayer()
    x = data.tokens(layer.C)
    opt = Adam(layer.w, rate)
    losses = []
    for i in range(steps):
        p = layer.forward(x, data.positions, data.docs)
        loss, dp = data.loss(p)
        losses.append(loss)
        if report and (i % 10 == 0 or i == steps - 1):
            report("step %d: loss %.2f" % (i, loss))
        opt.step(layer.backward(dp))
    return losses, layer


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 100, report=lambda s: print(s, flush=True))
