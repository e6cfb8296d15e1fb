"""Slot embeddings and the embedding table's gradient on the GPU vs the fp64 oracle ("DFlash
Draft Body", How It Works step 2).

Tolerances.  The forward rounds scale * e once in fp32 and once to the output's type:
(2^-24 + 2^-9 bf16 half step at its largest, 2^-8 relative at the smallest mantissa) --
2^-8 + 2^-24 relative for bf16, 2^-24 + 2^-24 (scale itself rounded to fp32) for fp32.  The
gradient adds n slots in fp32, at most n roundings of a partial sum bounded by sum |g|:
n 2^-24 sum |g|, then scale, the product and (accumulate) one addition: 4 * 2^-24, then the
table's type."""
import math

import numpy as np
import pytest

from oracle import dflash_oracle as orc

pytestmark = pytest.mark.gpu


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _half(name):
    return 2.0 ** -8 if name == "bf16" else 2.0 ** -24


def _guarded(shape, dtype, fill=3.0):
    """A tensor with 256 guard elements on both sides, filled."""
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 512,), fill, dtype=dtype, device="cuda")
    return buf, buf[256:256 + n].view(*shape)


def _guards_ok(buf, fill=3.0):
    return bool((buf[:256] == fill).all() and (buf[-256:] == fill).all())


def _ids(rng, T, V, kind):
    if kind == "blocks":        # anchor tokens and the mask token V - 1, some empty slots
        ids = np.where(np.arange(T) % 16 == 0, rng.integers(0, V, T), V - 1)
        ids[rng.random(T) < 0.1] = -1
    elif kind == "one":
        ids = np.full(T, rng.integers(0, V))
    elif kind == "none":
        ids = np.full(T, -1)
    elif kind == "runs":        # run lengths around the chunk sizes
        ids = np.repeat(rng.integers(0, V, T // 17 + 1), 17)[:T]
        rng.shuffle(ids[:T // 2])
    else:
        ids = rng.integers(-1, V, T)
    return ids.astype(np.int32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 5, 4096), (16, 1000, 256), (33, 77, 1001),
                                   (700, 5000, 8), (513, 300, 4096), (129, 64, 2050),
                                   (5, 11, 70000)])
def test_forward(lib, T, V, D, dtype):
    import torch
    import block_draft_model_proj_gb300 as dflash
    rng = np.random.default_rng(T + D)
    table = torch.as_tensor(rng.standard_normal((V, D)).astype(np.float32)).cuda().to(_dt(dtype))
    for kind, scale in (("blocks", 1.0), ("any", math.sqrt(D)), ("none", 2.0)):
        ids = _ids(rng, T, V, kind)
        buf, out = _guarded((T, D), table.dtype)
        dflash.dflash_embed_tokens(table, torch.as_tensor(ids).cuda(), out, scale=scale)
        dflash.dflash_device_status()
        ref = orc.embed_tokens(table.double().cpu().numpy(), ids, scale)
        got = out.double().cpu().numpy()
        assert _guards_ok(buf)
        assert np.all(got[ids < 0] == 0)
        assert np.all(np.abs(got - ref) <= (_half(dtype) + 2 * 2.0 ** -24) * np.abs(ref))
        if scale == 1.0:
            assert np.array_equal(got, ref)   # a gather


@pytest.mark.parametrize("table_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 9, 512), (16, 1000, 256), (37, 50, 1001),
                                   (700, 5000, 8), (1025, 40, 2052), (3000, 200, 520),
                                   (4096, 17, 24)])
@pytest.mark.parametrize("kind", ["blocks", "one", "none", "runs", "any"])
def test_gradient(lib, T, V, D, kind, dtype, table_dtype):
    import torch
    import block_draft_model_proj_gb300 as dflash
    rng = np.random.default_rng(T * 7 + D)
    g = torch.as_tensor(rng.standard_normal((T, D)).astype(np.float32)).cuda().to(_dt(dtype))
    ids = _ids(rng, T, V, kind)
    dev_ids = torch.as_tensor(ids).cuda()
    scale = 0.37
    g64 = g.double().cpu().numpy()
    ref = orc.embed_tokens_grad(g64, ids, V, scale)
    mag = orc.embed_tokens_grad(np.abs(g64), ids, V, scale)
    n = np.bincount(ids[ids >= 0], minlength=V)[:, None]
    for accumulate in (False, True):
        buf, out = _guarded((V, D), _dt(table_dtype))
        base = np.zeros((V, D))
        if accumulate:
            b = torch.as_tensor(rng.standard_normal((V, D)).astype(np.float32)).cuda().to(out.dtype)
            out.copy_(b)
            base = b.double().cpu().numpy()
        dflash.dflash_embed_tokens_grad(g, dev_ids, out, scale=scale, accumulate=accumulate)
        dflash.dflash_device_status()
        got = out.double().cpu().numpy()
        assert _guards_ok(buf)
        assert np.array_equal(got[n[:, 0] == 0], base[n[:, 0] == 0])
        want = base + ref
        tol = (n + 4) * 2.0 ** -24 * (mag + np.abs(base))
        tol = tol + _half(table_dtype) * (np.abs(want) + tol)
        assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))


@pytest.mark.parametrize("T", [8191, 8192, 8193, 16385, 40000, 70001])
@pytest.mark.parametrize("V", [300, 151936, 600000])
def test_gradient_of_many_slots(lib, T, V):
    """Both ways of sorting, one to three digits of the token."""
    import torch
    import block_draft_model_proj_gb300 as dflash
    rng = np.random.default_rng(T)
    D = 8
    ids = _ids(rng, T, V, "blocks")
    g = torch.as_tensor(rng.standard_normal((T, D)).astype(np.float32)).cuda()
    out = torch.full((V, D), math.nan, device="cuda")
    dflash.dflash_embed_tokens_grad(g, torch.as_tensor(ids).cuda(), out)
    dflash.dflash_device_status()
    g64 = g.double().cpu().numpy()
    ref, mag = np.zeros((V, D)), np.zeros((V, D))
    live = ids >= 0
    np.add.at(ref, ids[live], g64[live])
    np.add.at(mag, ids[live], np.abs(g64[live]))
    n = np.bincount(ids[live], minlength=V)[:, None]
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.all(err <= (n + 4) * 2.0 ** -24 * mag + 2.0 ** -24 * np.abs(ref))


def test_gradient_by_differences(lib):
    """d/dtable of sum(c * embed(table)) through the two calls: the forward is linear, so the
    difference of two tables gives the gradient's inner product with their step exactly, up to
    rounding: T * D terms of 2^-22 relative each."""
    import torch
    import block_draft_model_proj_gb300 as dflash
    rng = np.random.default_rng(31)
    T, V, D, scale = 300, 40, 96, 1.5
    ids = torch.as_tensor(_ids(rng, T, V, "blocks")).cuda()
    table, step = (torch.as_tensor(rng.standard_normal((V, D)).astype(np.float32)).cuda()
                   for _ in range(2))
    c = torch.as_tensor(rng.standard_normal((T, D)).astype(np.float32)).cuda()
    outs = []
    for t in (table + step, table - step):
        o = torch.empty((T, D), device="cuda")
        dflash.dflash_embed_tokens(t.contiguous(), ids, o, scale=scale)
        outs.append(o.double())
    grad = torch.empty((V, D), device="cuda")
    dflash.dflash_embed_tokens_grad(c, ids, grad, scale=scale)
    num = float(((outs[0] - outs[1]) * c.double()).sum() / 2)
    ana = float((grad.double() * step.double()).sum())
    size = float(((outs[0].abs() + outs[1].abs()) * c.double().abs()).sum())
    assert abs(num - ana) <= 2.0 ** -20 * size


def test_tokens_out_of_range(lib):
    import torch
    import block_draft_model_proj_gb300 as dflash
    V, D = 50, 64
    table = torch.randn((V, D), device="cuda")
    for T in (40, 20000):
        ids = torch.arange(T, dtype=torch.int32, device="cuda") % V
        g = torch.ones((T, D), device="cuda")
        want = torch.empty((V, D), device="cuda")
        clean = ids.clone()
        clean[3:9] = -1
        dflash.dflash_embed_tokens_grad(g, clean, want)
        dflash.dflash_device_status()
        ids[3:9] = torch.tensor([V, -2, 2**31 - 1, -2**31, V + 1, -3], device="cuda").int()
        out, grad = torch.full((T, D), 5.0, device="cuda"), torch.empty((V, D), device="cuda")
        dflash.dflash_embed_tokens(table, ids, out)
        with pytest.raises(RuntimeError, match="device index check"):
            dflash.dflash_device_status()
        assert not out[3:9].any() and torch.equal(out[9:], table[ids[9:].long()])
        dflash.dflash_embed_tokens_grad(g, ids, grad)
        with pytest.raises(RuntimeError, match="device index check"):
            dflash.dflash_device_status()
        assert torch.equal(grad, want)


def test_no_slots(lib):
    import torch
    import block_draft_model_proj_gb300 as dflash
    e = torch.empty
    ids = e(0, dtype=torch.int32, device="cuda")
    dflash.dflash_embed_tokens(torch.ones((3, 8), device="cuda"), ids, e((0, 8), device="cuda"))
    t = torch.ones((70, 8), device="cuda")
    dflash.dflash_embed_tokens_grad(e((0, 8), device="cuda"), ids, t, accumulate=True)
    assert (t == 1).all()
    dflash.dflash_embed_tokens_grad(e((0, 8), device="cuda"), ids, t)
    assert (t == 0).all()


def test_offsets_beyond_32_bits(lib):
    """A table of more than 2^31 elements: the last rows."""
    import torch
    import block_draft_model_proj_gb300 as dflash
    V, D = 300000, 8192
    table = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, 262144, 262143, V - 1], dtype=torch.int32, device="cuda")
    table[V - 1], table[262144], table[262143] = 3.0, 2.0, 1.0
    out = torch.empty((5, D), dtype=torch.bfloat16, device="cuda")
    dflash.dflash_embed_tokens(table, ids, out)
    assert out.float().mean(1).tolist() == [3.0, 0.0, 2.0, 1.0, 3.0]
    table.fill_(7.0)
    dflash.dflash_embed_tokens_grad(out, ids, table)
    dflash.dflash_device_status()
    assert table[V - 1].eq(6).all() and table[262144].eq(2).all() and table[262143].eq(1).all()
    assert int((table != 0).any(1).sum()) == 3


def test_same_bits_on_streams_and_in_graphs(lib):
    """The sums have one order: a captured graph, a side stream and a plain call agree bit for
    bit, and two graphs with workspaces of their own may run side by side."""
    import torch
    import block_draft_model_proj_gb300 as dflash
    rng = np.random.default_rng(33)
    V, D = 900, 264
    case = []
    for T in (3000, 18000):
        ids = torch.as_tensor(_ids(rng, T, V, "blocks")).cuda()
        g = torch.as_tensor(rng.standard_normal((T, D)).astype(np.float32)).cuda()
        want = torch.empty((V, D), device="cuda")
        dflash.dflash_embed_tokens_grad(g, ids, want)
        ws = dflash.workspace(dflash.dflash_embed_tokens_grad_workspace_size(V, D, T))
        case.append((g, ids, torch.empty_like(want), ws, want))
    torch.cuda.synchronize()

    def same():
        torch.cuda.synchronize()
        for c in case:
            assert torch.equal(c[2], c[4])
            c[2].fill_(math.nan)
        torch.cuda.synchronize()

    streams = [torch.cuda.Stream() for _ in case]
    for c, s in zip(case, streams):
        with torch.cuda.stream(s):
            dflash.dflash_embed_tokens_grad(c[0], c[1], c[2], ws=c[3])
    same()
    graphs = []
    for c in case:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            dflash.dflash_embed_tokens_grad(c[0], c[1], c[2], ws=c[3])
        graphs.append(gr)
    for _ in range(2):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        same()


def test_given_streams(lib):
    """A stream object or its handle; the workspace made for the call belongs to that stream."""
    import torch
    import block_draft_model_proj_gb300 as dflash
    rng = np.random.default_rng(34)
    T, V, D = 2500, 700, 264
    ids = torch.as_tensor(_ids(rng, T, V, "blocks")).cuda()
    g = torch.as_tensor(rng.standard_normal((T, D)).astype(np.float32)).cuda()
    want = torch.empty((V, D), device="cuda")
    dflash.dflash_embed_tokens_grad(g, ids, want)
    emb = torch.empty((T, D), device="cuda")
    dflash.dflash_embed_tokens(want, ids, emb)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got, e = torch.zeros_like(want), torch.zeros_like(emb)
        s.wait_stream(torch.cuda.current_stream())
        dflash.dflash_embed_tokens_grad(g, ids, got, stream=stream)
        dflash.dflash_embed_tokens(got, ids, e, stream=stream)
        junk = torch.full((1 << 20,), 7.0, device="cuda")   # would take a freed workspace's place
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(e, emb) and junk.eq(7).all()


def _walk_ids(rng, T, V, kind):
    """Tokens whose changes fall on every place of a walk over consecutive slots."""
    if kind == "few":           # two or three tokens in all: repeats and changes anywhere
        return rng.integers(0, min(V, 3), T).astype(np.int32)
    if kind == "text":          # plain text: a frequent token among others
        return np.where(rng.random(T) < 0.5, 7 % V, rng.integers(0, V, T)).astype(np.int32)
    ids = np.where(np.arange(T) % kind == 0, rng.integers(0, V, T), V - 1)
    ids[rng.random(T) < 0.05] = -1      # single empty slots
    return ids.astype(np.int32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [3, 5, 6, 7, 10, 16, "few", "text"])
@pytest.mark.parametrize("T,V,D", [(2600, 300, 4096), (8195, 900, 4096), (2600, 300, 1001),
                                   (1003, 40, 2050), (20011, 500, 520)])
def test_forward_of_long_walks(lib, T, V, D, kind, dtype):
    """Enough slots that a row of threads takes many consecutive ones (up to 16), whose rows
    stay in its registers while the token repeats."""
    import torch
    import block_draft_model_proj_gb300 as dflash
    rng = np.random.default_rng(T + D)
    table = torch.as_tensor(rng.standard_normal((V, D)).astype(np.float32)).cuda().to(_dt(dtype))
    ids = torch.as_tensor(_walk_ids(rng, T, V, kind)).cuda()
    rows = table.double()[ids.long().clamp(min=0)] * (ids >= 0)[:, None]
    for scale in (1.0, 1.7):
        buf, out = _guarded((T, D), table.dtype)
        dflash.dflash_embed_tokens(table, ids, out, scale=scale)
        dflash.dflash_device_status()
        assert _guards_ok(buf)
        wrong = (out.double() - scale * rows).abs() > \
            (0.0 if scale == 1.0 else _half(dtype) + 2 * 2.0 ** -24) * (scale * rows).abs()
        assert not wrong.any(), wrong.any(1).nonzero()[:8, 0].tolist()


def test_the_most_slots(lib):
    """2^31 - 1 slots: the last chunk's, tile's and CTA's ends lie at the end of the int range."""
    import torch
    import block_draft_model_proj_gb300 as dflash
    T, V = 2**31 - 1, 5
    table = torch.arange(1, V + 1, device="cuda").to(torch.bfloat16).view(V, 1)
    ids = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
    ids[-3:] = torch.tensor([4, -1, 2], dtype=torch.int32, device="cuda")
    out = torch.full((T, 1), 9.0, dtype=torch.bfloat16, device="cuda")
    dflash.dflash_embed_tokens(table, ids, out)
    dflash.dflash_device_status()
    assert out[-3:, 0].tolist() == [5.0, 0.0, 3.0]
    for i in range(0, T, 1 << 28):
        e = min(T, i + (1 << 28))
        assert torch.equal(out[i:e, 0], (ids[i:e] + 1).to(torch.bfloat16))
    at = torch.cat([torch.tensor([0, T - 3, T - 2, T - 1], device="cuda"),
                    torch.randint(0, T, (1000,), device="cuda")]).unique()
    out.zero_()
    out[at] = 1.0
    grad = torch.full((V, 1), math.nan, device="cuda")
    dflash.dflash_embed_tokens_grad(out, ids, grad)
    dflash.dflash_device_status()
    hit = ids[at]
    assert torch.equal(grad[:, 0], torch.bincount(hit[hit >= 0], minlength=V).float())
