"""examples/moe_block.py: every stage of a decode step against its formula in 64
bits, from the stage's own inputs."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.double().cpu().numpy()


def expert_ffn(blob, H, I, x, ex):
    """W_d (silu(W_g x) * W_u x) of an NVFP4 blob (bytes on the host)."""
    code, scale, glob = ex.bank_offsets(H, I)
    g = blob[glob:glob + 12].view(np.float32)
    mats = []
    for i, (n, k) in enumerate(((I, H), (I, H), (H, I))):
        c = blob[code[i]:code[i] + n * k // 2].reshape(n, k // 2)
        s = blob[scale[i]:scale[i] + n * k // 16].reshape(n, k // 16)
        mats.append(ref.decode(c, s, True, g[i]))
    a, u = mats[0] @ x, mats[1] @ x
    return mats[2] @ (a / (1 + np.exp(-a)) * u)


@pytest.mark.parametrize("rows", [1, 5])
def test_every_stage_of_a_step(rows):
    ex = example()
    H, I, E, k = 1024, 512, 16, 2
    d = ex.Decoder(n_layers=2, n_experts=E, top_k=k, hidden=H, inter=I, vocab=1000, n_slots=24, rows=rows)
    tokens = torch.arange(rows, device="cuda") * 7
    seen = []

    def trace(layer, dec):
        torch.cuda.synchronize()
        keep = {n: f64(getattr(dec, n)) for n in ("h", "x", "y", "z", "w", "logits")}
        keep.update(ids=dec.ids.cpu().numpy(), xc=dec.xc.cpu().numpy(), xs=dec.xs.cpu().numpy())
        seen.append(keep)

    for step in range(3):
        seen.clear()
        nxt = d.step(tokens, trace)
        # the first pre-norm
        h, x, _ = ref.block_norm(f64(d.embed[tokens]), pre_w=f64(d.pre[0]), eps=float(np.float32(1e-6)))
        assert np.array_equal(seen[0]["h"], h)
        assert np.allclose(seen[0]["x"], x, rtol=2.0 ** -8 * 1.01, atol=1e-6)
        for layer in range(2):
            s, after = seen[layer], seen[layer + 1]
            z = s["x"] @ f64(d.router[layer]).T
            assert np.abs(s["z"] - z).max() < 1e-4
            ids, w, gap = ref.route(s["z"], k, score="sigmoid", bias=f64(d.bias[layer]), groups=4,
                                    topk_groups=2, group_top=2, scale=2.5)
            assert gap < 1e-6 or np.array_equal(ids, s["ids"])
            if np.array_equal(ids, s["ids"]):
                assert np.allclose(s["w"], w, rtol=64 * 2.0 ** -24, atol=0)
            y = np.zeros((rows, H))
            for b in range(rows):
                for j in range(k):
                    e = int(s["ids"][b, j])
                    y[b] += s["w"][b, j] * expert_ffn(d.blobs[layer * E + e].numpy(), H, I, s["x"][b], ex)
            # the layer's own tolerance for 4-bit experts
            assert (np.abs(s["y"] - y) <= 2e-2 + 1e-2 * np.abs(y)).all()
            h, x, size = ref.block_norm(s["h"], s["y"], f64(d.post[layer]), f64(d.gate[layer]), "sigmoid", 0.5,
                                        f64(d.pre[layer + 1]), eps=float(np.float32(1e-6)))
            assert (np.abs(after["h"] - h) <= 32 * 2.0 ** -24 * size).all()
            assert np.allclose(after["x"], x, rtol=2.0 ** -8 * 1.01, atol=1e-5)
        last = seen[2]
        xc, xs = ref.quantize(last["x"].astype(np.float32), True, d.x_g.item())
        assert np.array_equal(last["xc"], xc) and np.array_equal(last["xs"], xs)
        a = ref.decode(xc, xs, True, d.x_g.item())
        w = ref.decode(d.head_c.cpu().numpy(), d.head_s.cpu().numpy(), True, d.head_g.item())
        err = np.abs(last["logits"] - a @ w.T)
        assert (err <= (H / 32 + 40) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T) + 2.0 ** -23 * np.abs(a @ w.T)).all()
        assert np.array_equal(nxt.cpu().numpy(), last["logits"].argmax(1))
        tokens = nxt
    assert sum(d.cache.stats(layer)["calls"] for layer in range(2)) == 6
