"""A decoder layer's calls run together, forward and back: positions and norms of q and k, windowed attention over the
tokens themselves, the residual step, the reading of an encoder's states by cross attention, the second residual step. Every
stored result is held against its definition in 64 bits from the stored tensors before it, under the tolerances of that
operator's own tests, eagerly and after replays of a captured graph."""
import pytest
import torch

import vision_encoder_varlen_gb300 as vit
import test_gpu_cross_attn as cross
import test_gpu_cross_attn_bwd as cross_back
import test_gpu_mrope as rope
import test_gpu_norm_residual as norm
import test_gpu_window_attn as own
import test_gpu_window_attn_bwd as own_back

pytestmark = pytest.mark.gpu
EPS = 1e-6


class Layer:
    def __init__(self, ql, kl, Hq, Hk, D, window, sinks):
        g = torch.Generator(device="cuda").manual_seed(21)
        bf = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
        self.T, self.C, self.shape = sum(ql), Hq * D, (sum(ql), Hq, D)
        self.Hq, self.Hk, self.mask = Hq, Hk, (window, sinks)
        self.bounds, self.reading = (max(ql), max(ql)), (max(ql), max(kl))
        self.qkv, self.x, self.q2 = bf(self.T, Hq + 2 * Hk, D), bf(self.T, self.C), bf(*self.shape)
        self.states = bf(sum(kl), 2 * Hk, D)
        self.dz, self.dh = bf(self.T, self.C), bf(self.T, self.C)
        self.w, self.w1, self.w2 = (1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")).bfloat16(), bf(self.C), bf(self.C)
        self.freq = (1e4 ** (-torch.arange(D // 2, device="cuda").double() / (D // 2))).float()
        self.pos = torch.cat([torch.arange(m) for m in ql]).int().cuda()[:, None].expand(self.T, 3).contiguous()
        self.sec, self.cu, self.cu_s = (D // 2 - 8, 4, 4), own.offsets(ql), own.offsets(kl)
        self.s = {}

    def run(self):
        s, Hq, Hk, flat = self.s, self.Hq, self.Hk, (self.T, self.C)
        raw, k2, v2 = self.qkv, self.states[:, :Hk], self.states[:, Hk:]
        s["q"], s["k"] = vit.qk_norm_mrope(raw[:, :Hq], raw[:, Hq:Hq + Hk], self.pos, self.freq, self.sec, self.w, EPS)
        v = raw[:, Hq + Hk:]
        s["y"], s["lse"] = vit.window_attn(s["q"], s["k"], v, self.cu, self.cu, *self.bounds, *self.mask, return_lse=True)
        s["h"], s["z"] = vit.norm_residual(self.x, s["y"].view(flat), w_pre=self.w1, eps=EPS)
        s["y2"], s["lse2"] = vit.cross_attn(self.q2, k2, v2, self.cu, self.cu_s, *self.reading, return_lse=True)
        s["h2"], s["z2"] = vit.norm_residual(s["h"], s["y2"].view(flat), w_pre=self.w2, eps=EPS)
        # and back
        s["dh"], s["dy2"], _, _, s["dw2"] = vit.norm_residual_bwd(self.dz, self.dh, s["h2"], s["y2"].view(flat), w_pre=self.w2,
                                                                 eps=EPS)
        s["dq2"], s["dk2"], s["dv2"] = vit.cross_attn_bwd(s["dy2"].view(self.shape), self.q2, k2, v2, s["y2"], s["lse2"],
                                                          self.cu, self.cu_s, *self.reading)
        s["dx"], s["dy"], _, _, s["dw1"] = vit.norm_residual_bwd(self.dz, s["dh"], s["h"], s["y"].view(flat), w_pre=self.w1,
                                                                eps=EPS)
        s["dq"], s["dk"], s["dv"] = vit.window_attn_bwd(s["dy"].view(self.shape), s["q"], s["k"], v, s["y"], s["lse"], self.cu,
                                                        self.cu, *self.bounds, *self.mask)
        s["dq0"], s["dk0"], s["dnorm"] = vit.qk_norm_mrope_bwd(s["dq"], s["dk"], raw[:, :Hq], raw[:, Hq:Hq + Hk], self.pos,
                                                               self.freq, self.sec, self.w, EPS)

    def check(self):
        s, Hq, Hk = self.s, self.Hq, self.Hk
        raw, k2, v2 = self.qkv, self.states[:, :Hk], self.states[:, Hk:]
        a, halves = rope.angles(self.pos, self.freq, self.sec, False), (raw[:, :Hq], raw[:, Hq:Hq + Hk])
        for row, (name, x) in enumerate(zip("qk", halves)):
            rope.close(s[name], *rope.reference(x, self.w[row], a, False, EPS), name)
        v = raw[:, Hq + Hk:]
        own.check(s["y"], s["lse"], own.reference(s["q"], s["k"], v, self.cu, self.cu, None, *self.mask))
        self.step(self.x, s["y"], self.w1, s["h"], s["z"])
        cross.check(s["y2"], s["lse2"], cross.reference(self.q2, k2, v2, self.cu, self.cu_s))
        self.step(s["h"], s["y2"], self.w2, s["h2"], s["z2"])
        self.step_back(self.dh, s["h2"], self.w2, s["dh"], s["dy2"], s["dw2"])
        cross_back.check((s["dq2"], s["dk2"], s["dv2"]),
                         cross_back.reference(self.q2, k2, v2, s["dy2"].view(self.shape), self.cu, self.cu_s))
        self.step_back(s["dh"], s["h"], self.w1, s["dx"], s["dy"], s["dw1"])
        own_back.check((s["dq"], s["dk"], s["dv"]), own_back.reference(s["q"], s["k"], v, s["dy"].view(self.shape), self.cu,
                                                                       self.cu, None, *self.mask))
        for row, (d, got, x) in enumerate((("dq", "dq0", halves[0]), ("dk", "dk0", halves[1]))):
            ref, mag, sw, mw = rope.reference_grad(s[d], x, self.w[row], a, False, EPS)
            rope.close(s[got], ref, mag, got)
            tol = ((self.T * x.shape[1] + 64) * 2.0 ** -24 + 2.0 ** -18) * mw
            assert ((s["dnorm"][row].double() - sw).abs() <= tol).all()

    def step(self, x, y, w, h, z):
        X, Y = x.double(), y.view(self.T, self.C).double()
        H, mag = X + Y, X.abs() + Y.abs()
        norm.close(h, H, mag, "h")
        r = norm.rms(H)
        norm.close(z, H * r * w.double(), 2 * (mag + H.abs()) * r * w.double().abs(), "z")

    def step_back(self, dh, h, w, dx, dy, dw):
        H = h.double()
        r = norm.rms(H)
        hh, dn = H * r, self.dz.double() * w.double()
        dH = dh.double() + r * (dn - hh * (dn * hh).mean(-1, keepdim=True))
        mag = dh.double().abs() + r * (dn.abs() + hh.abs() * (dn * hh).abs().mean(-1, keepdim=True))
        norm.close(dx, dH, mag, "dx")
        norm.close(dy, dH, mag, "dy")
        terms = self.dz.double() * hh
        assert ((dw.double() - terms.sum(0)).abs() <= ((self.T + 64) * 2.0 ** -24 + norm.F32) * terms.abs().sum(0)).all()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("ql,kl,Hq,Hk,D,window,sinks", [([150, 37, 1], [400, 1, 77], 8, 2, 64, 40, 4),
                                                        ([300], [1000], 4, 4, 80, 128, 0),
                                                        ([1] * 5, [900, 3, 64, 65, 1], 16, 2, 128, 7, 1)])
def test_each_result(ql, kl, Hq, Hk, D, window, sinks, captured):
    layer = Layer(ql, kl, Hq, Hk, D, window, sinks)
    layer.run()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.run()
        for t in (layer.qkv, layer.x, layer.q2, layer.dz):     # other values of the same shapes
            t.copy_(t.flip(0))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
    layer.check()
