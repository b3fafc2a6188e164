"""The 8-bit LM head and the block quantiser on the GPU against their definitions
(oracle/losses.py). Needs a GB300.

Quantised codes and scales follow from single fp32 operations, so they are equal
bit for bit. A logit is a sum of K exact products (an e4m3 product has 8
significant bits) in fp32, whose additions may truncate (2^-23 of the magnitudes
that they add), a scale product (2^-24) and a scaled addition (2^-24) for each
block, and one rounding to the logits' type."""
import numpy as np
import pytest

import oracle.losses as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sampler():
    from decode_step_token_gb300 import build
    build.build_library()
    import decode_step_token_gb300 as d
    s = d.Sampler(max_rows=1024, max_vocab=262144)
    yield s
    s.close()


def _source(rng, rows, cols, kind):
    import torch

    x = (rng.standard_normal((rows, cols)) * np.exp(1.5 * rng.standard_normal(cols))).astype(np.float32)
    if rows > 2:
        x[1] = 0
        x[2] *= np.float32(1e-33)
    t = torch.from_numpy(x)
    t = t.to(torch.bfloat16) if kind == "bf16" else t
    return t, t.float().numpy()


@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (3, 127, 0, 0), (2, 128, 0, 0), (5, 129, 1, 1),
                                                 (129, 300, 5, 3), (128, 256, 0, 0), (257, 1000, 8, 8),
                                                 (64, 4096, 0, 0), (1000, 4100, 4, 0), (300, 777, 0, 1)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("height", [1, 128])
def test_quantize(sampler, rows, cols, pad, shift, kind, height):
    import torch

    rng = np.random.default_rng(rows * 1000 + cols)
    t, x = _source(rng, rows, cols, kind)
    flat = torch.full((rows * (cols + pad) + shift + 64,), float("nan"), dtype=t.dtype, device="cuda:0")
    src = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    src.copy_(t)
    up, across = -(-rows // height), -(-cols // 128)
    vflat = torch.full((rows * (cols + pad) + shift + 64,), 0x55, dtype=torch.uint8, device="cuda:0")
    values = vflat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    scales = torch.full((up, across + 2), -7.0, device="cuda:0")
    sampler.quantize_blocks(src=src, block_rows=height, out_values=values.view(torch.float8_e4m3fn),
                            out_scales=scales)
    codes, want = L.quantize(x, height)
    np.testing.assert_array_equal(scales[:, :across].cpu().numpy(), want)
    got = values.cpu().numpy()
    # a zero's sign is kept, so the codes are equal as they are
    np.testing.assert_array_equal(got, codes)
    assert (scales[:, across:] == -7).all()
    values.fill_(0x55)
    assert (vflat == 0x55).all(), "written beside the values"


@pytest.mark.parametrize("height", [1, 128])
def test_quantize_what_is_not_finite(sampler, height):
    import torch

    x = torch.randn((200, 400), device="cuda:0")
    x[3, 5], x[150, 390], x[7, 130] = float("nan"), float("inf"), -float("inf")
    values = torch.empty((200, 400), dtype=torch.float8_e4m3fn, device="cuda:0")
    scales = torch.empty((-(-200 // height), 4), device="cuda:0")
    sampler.quantize_blocks(src=x, block_rows=height, out_values=values, out_scales=scales)
    codes, want = L.quantize(x.cpu().numpy(), height)
    np.testing.assert_array_equal(scales.cpu().numpy(), want)
    np.testing.assert_array_equal(values.view(torch.uint8).cpu().numpy(), codes)


def _head(seed, rows, V, K):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (rows + V, K)).astype(np.uint8)
    codes[codes & 127 == 127] = 0  # no NaN
    h, w = codes[:rows], codes[rows:]
    g = -(-K // 128)
    sh = rng.uniform(0.001, 0.01, (rows, g)).astype(np.float32)
    sw = (rng.uniform(0.5, 1.0, (-(-V // 128), g)) / np.sqrt(K)).astype(np.float32)
    return h, sh, w, sw


def _up(a, stride=None, fill=0x7f):
    """Codes on the device with rows `stride` apart; what lies between is NaN."""
    import torch

    rows, K = a.shape
    stride = stride or -(-K // 16) * 16
    t = torch.full((rows, stride), fill, dtype=torch.uint8, device="cuda:0")
    t[:, :K] = torch.from_numpy(a).to("cuda:0")
    return t[:, :K]


def _close(got, want, mag, K, kind):
    # K truncating additions inside the blocks, a product and an addition for each of the blocks
    g = -(-K // 128)
    bound = (min(K, 128) * 2.0 ** -23 + (2 + g) * 2.0 ** -24) * mag
    half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -24
    bad = np.abs(got - want) > half * np.abs(want) + (1 + half) * bound
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 129, 130), (3, 1000, 64), (16, 4096, 256), (17, 300, 1000), (31, 5003, 96),
          (64, 2000, 512), (65, 257, 129), (127, 640, 384), (128, 1024, 1024), (129, 1025, 300), (200, 3001, 256),
          (255, 511, 200), (256, 256, 4096), (257, 1300, 640), (513, 900, 16), (700, 1111, 1000),
          # few tiles with many blocks of K
          (1, 1, 600), (16, 1000, 4096), (32, 2000, 3000), (8, 2000, 8192), (5, 4000, 2500), (20, 9001, 1024),
          (40, 3000, 4100), (64, 500, 1900), (100, 5000, 2048), (128, 130, 1030), (33, 1921, 4096),
          # several tiles for each CTA and pair, with more than one ring's blocks
          (140, 42000, 1300), (300, 21000, 640), (600, 20003, 384), (40, 40011, 2100)]


@pytest.mark.parametrize("rows,V,K", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_product(sampler, rows, V, K, kind):
    import torch

    h, sh, w, sw = _head(rows * 7 + V, rows, V, K)
    ldl = V + 3
    out = torch.full((rows, ldl), -7.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda:0")
    hs = torch.full((rows, sh.shape[1] + 1), float("nan"), device="cuda:0")
    ws = torch.full((sw.shape[0], sw.shape[1] + 2), float("nan"), device="cuda:0")
    hs[:, :-1], ws[:, :-2] = torch.from_numpy(sh).cuda(), torch.from_numpy(sw).cuda()
    sampler.lm_head_scaled(hidden=_up(h), hidden_scale=hs, weight=_up(w, -(-K // 16) * 16 + 32), weight_scale=ws,
                           logits=out)
    got = out.double().cpu().numpy()
    assert (got[:, V:] == -7).all(), "written beside the logits"
    want, mag = L.scaled_head(h, sh, w, sw)
    _close(got[:, :V], want, mag, K, kind)


def test_full_size_columns(sampler):
    """64 and 1000 rows x 128000 x 4096: sampled columns against the definition."""
    import torch

    V, K = 128000, 4096
    gen = torch.Generator(device="cuda:0").manual_seed(3)
    w = (100 * torch.randn((V, K), generator=gen, device="cuda:0")).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand((1000, 32), generator=gen, device="cuda:0") + 0.5
    cols = np.random.default_rng(0).choice(V, 600, replace=False)
    cols[:3] = 0, 127, V - 1
    for rows in (64, 1000):
        h = (100 * torch.randn((rows, K), generator=gen, device="cuda:0")).clamp(-448, 448).to(torch.float8_e4m3fn)
        hs = torch.rand((rows, 32), generator=gen, device="cuda:0") * 1e-4
        out = torch.empty((rows, V), dtype=torch.bfloat16, device="cuda:0")
        sampler.lm_head_scaled(hidden=h, hidden_scale=hs, weight=w, weight_scale=ws, logits=out)
        wc = w.view(torch.uint8)[torch.from_numpy(cols).cuda()].cpu().numpy()
        t = L.e4m3_table()
        H = t[h.view(torch.uint8).cpu().numpy()] * np.repeat(hs.double().cpu().numpy(), 128, 1)
        W = t[wc] * np.repeat(ws.double().cpu().numpy()[cols // 128], 128, 1)
        _close(out[:, torch.from_numpy(cols).cuda()].double().cpu().numpy(), H @ W.T, np.abs(H) @ np.abs(W).T, K,
               "bf16")


def test_what_is_not_finite_stays_in_its_row(sampler):
    import torch

    rows, V, K = 20, 700, 512
    h, sh, w, sw = _head(9, rows, V, K)
    h[3, 200] = 0x7f
    sh[5, 1] = np.nan
    out = torch.empty((rows, V), device="cuda:0")
    sampler.lm_head_scaled(hidden=_up(h), hidden_scale=torch.from_numpy(sh).cuda(), weight=_up(w),
                           weight_scale=torch.from_numpy(sw).cuda(), logits=out)
    got = out.cpu().numpy()
    nan = np.isnan(got).all(1)
    assert nan.nonzero()[0].tolist() == [3, 5] and np.isfinite(got[~nan]).all()


def _step(sampler, rows, V, K, kind):
    """Quantise, make the logits and sample greedily and at T = 0.8, through the chained entry."""
    import torch

    gen = torch.Generator(device="cuda:0").manual_seed(11)
    x = torch.randn((rows, K), generator=gen, device="cuda:0").to(torch.bfloat16)
    w = (torch.randn((V, K), generator=gen, device="cuda:0") * 0.1).to(torch.bfloat16)
    q = [torch.empty(t.shape, dtype=torch.float8_e4m3fn, device="cuda:0") for t in (x, w)]
    s = [torch.empty((rows, -(-K // 128)), device="cuda:0"), torch.empty((-(-V // 128), -(-K // 128)), device="cuda:0")]
    sampler.quantize_blocks(src=x, block_rows=1, out_values=q[0], out_scales=s[0])
    sampler.quantize_blocks(src=w, block_rows=128, out_values=q[1], out_scales=s[1])
    op = dict(hidden=q[0], hidden_scale=s[0], weight=q[1], weight_scale=s[1])
    dt = torch.bfloat16 if kind == "bf16" else torch.float32
    apart, chained = torch.empty((rows, V), dtype=dt, device="cuda:0"), torch.empty((rows, V), dtype=dt, device="cuda:0")
    T = torch.where(torch.arange(rows, device="cuda:0") % 2 == 0, 0.0, 0.8)
    tok = [torch.full((rows,), -7, dtype=torch.int32, device="cuda:0") for _ in range(2)]
    sampler.lm_head_scaled(logits=apart, **op)
    sampler.sample(logits=apart, temperature=T, out_tokens=tok[0])
    args = sampler.make_args(logits=chained, temperature=T, out_tokens=tok[1])
    sampler.lm_head_scaled_sample_args(args, **op)
    return apart, chained, tok, (args, op, T)


@pytest.mark.parametrize("rows,V,K,kind", [(1, 5000, 256, "bf16"), (64, 20000, 1024, "bf16"), (33, 9001, 400, "f32"),
                                           (300, 4000, 512, "bf16")])
def test_chained_to_the_sampler(sampler, rows, V, K, kind):
    import torch

    apart, chained, tok, _ = _step(sampler, rows, V, K, kind)
    assert torch.equal(apart, chained) and torch.equal(tok[0], tok[1])
    greedy = torch.arange(rows, device="cuda:0") % 2 == 0
    assert torch.equal(tok[1][greedy].long(), apart.float().argmax(1)[greedy])


def test_graph_replay(sampler):
    import torch

    apart, chained, tok, (args, op, _) = _step(sampler, 48, 16000, 512, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sampler.lm_head_scaled_sample_args(args, stream=torch.cuda.current_stream().cuda_stream, **op)
    chained.zero_()
    tok[1].fill_(-7)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(apart, chained) and torch.equal(tok[0], tok[1])


def test_refusals(sampler):
    import torch
    import decode_step_token_gb300 as d

    h, sh, w, sw = _head(12, 4, 300, 64)
    op = dict(hidden=_up(h), hidden_scale=torch.from_numpy(sh).cuda(), weight=_up(w),
              weight_scale=torch.from_numpy(sw).cuda())
    out = torch.empty((4, 300), device="cuda:0")

    def code(**kw):
        with pytest.raises(d.SamplerError) as e:
            sampler.lm_head_scaled(**{**op, "logits": out, **kw})
        return e.value.code

    assert code(hidden=_up(h, 72)) == -2                             # a stride off 16
    assert code(weight=_up(np.zeros((301, 65), np.uint8))[1:, 1:]) == -2   # a start off 16
    with pytest.raises(ValueError, match="logits"):
        sampler.lm_head_scaled(**{**op, "logits": out[:3]})
    with pytest.raises(ValueError, match="weight_scale"):
        sampler.lm_head_scaled(**{**op, "weight_scale": op["weight_scale"][:2], "logits": out})
    with pytest.raises(ValueError, match="columns"):
        sampler.lm_head_scaled(**{**op, "hidden": op["hidden"][:, :63], "logits": out})
    x = torch.zeros((4, 64), device="cuda:0")
    for rows in (0, 2, 127):
        with pytest.raises(d.SamplerError) as e:
            sampler.quantize_blocks(src=x, block_rows=rows, out_values=op["hidden"],
                                    out_scales=torch.empty((4, 1), device="cuda:0"))
        assert e.value.code == -9
    assert sampler.stat(d.SAMPLER_STAT_LM_HEAD_TIMEOUTS) == 0
    empty = _up(np.zeros((0, 64), np.uint8))
    sampler.lm_head_scaled(**{**op, "hidden": empty, "hidden_scale": torch.empty((0, 1), device="cuda:0"),
                              "logits": out})


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V,K", [(7, 900, 300), (32, 30000, 4096), (33, 900, 300), (300, 20000, 640)])
def test_waits_that_give_up(sampler, rows, V, K, kind):
    """On a handle whose waits give up at once the head ends, counts every block and writes nothing; another handle
    is not affected."""
    import torch
    import decode_step_token_gb300 as d

    h, sh, w, sw = _head(21, rows, V, K)
    op = dict(hidden=_up(h), hidden_scale=torch.from_numpy(sh).cuda(), weight=_up(w),
              weight_scale=torch.from_numpy(sw).cuda())
    out = torch.full((rows, V), -7.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda:0")
    tiles = -(-V // 128) if rows <= 32 else -(-V // 256) * -(-rows // 128)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    with d.Sampler(max_rows=64, max_vocab=V, short_waits=True) as short:
        short.lm_head_scaled(logits=out, **op)
        assert short.stat(d.SAMPLER_STAT_LM_HEAD_TIMEOUTS, reset=True) == min(tiles, sms)
    assert (out == -7).all()
    sampler.lm_head_scaled(logits=out, **op)
    assert sampler.stat(d.SAMPLER_STAT_LM_HEAD_TIMEOUTS) == 0
    want, mag = L.scaled_head(h, sh, w, sw)
    _close(out.double().cpu().numpy(), want, mag, K, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("pad", ["none", "padded"])
@pytest.mark.parametrize("rows,V,K", [(33, 1000, 200), (65, 1032, 130), (129, 4104, 128), (300, 20000, 200),
                                      (64, 256, 300), (200, 264, 64), (45, 8, 128), (128, 513, 140), (333, 20011, 96),
                                      (160, 50257, 64), (513, 30004, 32)])
def test_logits_on_16_bytes(sampler, rows, V, K, pad, kind):
    """Rows of logits that lie on 16 bytes are stored by the TMA engine, whose boxes end where the logits do: at a last
    tile of the vocabulary that is cut off, or stored otherwise, and at the last rows. Nothing is written beside."""
    import torch

    h, sh, w, sw = _head(rows + V, rows, V, K)
    ldl = -(-V // 8) * 8 + (8 if pad == "padded" else 0)
    guard = 140  # rows after the last: more than a tile's
    out = torch.full((rows + guard, ldl), -7.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda:0")
    assert out.data_ptr() % 16 == 0 and ldl * out.element_size() % 16 == 0
    sampler.lm_head_scaled(hidden=_up(h), hidden_scale=torch.from_numpy(sh).cuda(), weight=_up(w),
                           weight_scale=torch.from_numpy(sw).cuda(), logits=out[:rows])
    assert (out[:, V:] == -7).all() and (out[rows:] == -7).all(), "written beside the logits"
    want, mag = L.scaled_head(h, sh, w, sw)
    _close(out[:rows, :V].double().cpu().numpy(), want, mag, K, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(2500, 4100, 4), (4801, 4200, 0), (20000, 1000, 1)])
def test_quantize_many_rows(sampler, rows, cols, pad, kind):
    """Rows for which a thread takes several; a block is one row here, so some of the rows are compared."""
    import torch

    gen = torch.Generator(device="cuda:0").manual_seed(rows)
    dt = torch.bfloat16 if kind == "bf16" else torch.float32
    src = torch.randn((rows, cols + pad), generator=gen, device="cuda:0", dtype=dt)[:, :cols]
    src[rows // 2, 300] = float("inf")
    values = torch.full((rows, cols + pad), 0x55, dtype=torch.uint8, device="cuda:0")
    scales = torch.empty((rows, -(-cols // 128)), device="cuda:0")
    sampler.quantize_blocks(src=src, block_rows=1, out_values=values[:, :cols].view(torch.float8_e4m3fn),
                            out_scales=scales)
    at = np.unique(np.concatenate([np.arange(5), [rows // 2], np.arange(rows - 70, rows),
                                   np.random.default_rng(0).integers(0, rows, 200)]))
    codes, want = L.quantize(src[torch.from_numpy(at).cuda()].float().cpu().numpy(), 1)
    np.testing.assert_array_equal(scales.cpu().numpy()[at], want)
    np.testing.assert_array_equal(values[:, :cols].cpu().numpy()[at], codes)
    assert (values[:, cols:] == 0x55).all(), "written beside the values"
