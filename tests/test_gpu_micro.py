"""Microscaled 4 bits on the GPU against their definitions (oracle/micro.py). Needs a GB300.

Codes, scales and row scales follow from exact steps, so they are equal bit for bit, and
so are values read back in double's reach (a code of 2 digits times a scale of 4 times a
power of two; otherwise one fp32 rounding for each of two products and one to the type).
A logit is a sum of K exact products (of 12 digits at most) in fp32, whose additions may
truncate (2^-23 of the magnitudes that they add), two products with the row scales (2^-24
each) and one rounding to the logits' type."""
import numpy as np
import pytest

import oracle.micro as M

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
    if rows > 4:
        x[1] = 0
        x[2] *= np.float32(1e-33)
        x[3] = rng.integers(-24, 25, cols)  # quotients halfway between codes
        x[4, cols // 2:] *= np.float32(1e-7)
    t = torch.from_numpy(x)
    t = t.to(torch.bfloat16) if kind == "bf16" else t
    return t, t.float().numpy()


def _quantize(sampler, src, block, stride=None):
    """(values, scales, row scales, the values' whole buffer) of a source on the device."""
    import torch

    rows, cols = src.shape
    half = (cols + 1) // 2
    stride = stride or -(-half // 16) * 16
    whole = torch.full((rows, stride), 0x55, dtype=torch.uint8, device="cuda:0")
    scales = torch.full((sampler.micro_scale_bytes(rows, cols, block) + 64,), 0x55, dtype=torch.uint8, device="cuda:0")
    row_scale = torch.full((rows + 3,), -7.0, device="cuda:0")
    sampler.quantize_micro(src=src, out_values=whole[:, :half], out_scales=scales, out_row_scale=row_scale, block=block)
    assert (scales[-64:] == 0x55).all() and (row_scale[rows:] == -7).all(), "written beside the scales"
    assert (whole[:, half:] == 0x55).all(), "written beside the values"
    return whole[:, :half], scales[:-64], row_scale[:rows]


@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (3, 15, 0, 0), (2, 16, 0, 0), (5, 33, 1, 1), (127, 64, 0, 0),
                                                 (129, 300, 5, 3), (128, 256, 0, 0), (257, 1000, 8, 8), (64, 4096, 0, 0),
                                                 (200, 4100, 4, 0), (300, 777, 0, 1), (9, 8192, 0, 0), (7, 16384, 0, 0),
                                                 (6, 16385, 1, 0), (5, 40001, 7, 8), (1000, 130, 0, 0)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
def test_quantize_and_back(sampler, rows, cols, pad, shift, kind, block):
    import torch

    rng = np.random.default_rng(rows * 1000 + cols)
    t, x = _source(rng, rows, cols, kind)
    flat = torch.full((rows * (cols + pad) + shift + 64,), float("nan"), dtype=t.dtype, device="cuda:0")
    src = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    src.copy_(t)
    half = (cols + 1) // 2
    got, scales, row_scale = _quantize(sampler, src, block, half + pad)
    codes, want_scales, want_row, values = M.quantize(x, block)
    np.testing.assert_array_equal(row_scale.cpu().numpy(), want_row)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_scales)
    np.testing.assert_array_equal(got.cpu().numpy(), codes)  # the zeros' signs, too
    for out_kind in (torch.bfloat16, torch.float32):
        whole = torch.full((rows, cols + pad), -7.0, dtype=out_kind, device="cuda:0")
        sampler.micro_rows(values=got, scales=scales, row_scale=row_scale, block=block, out=whole[:, :cols])
        assert (whole[:, cols:] == -7).all()
        want = torch.from_numpy(values.astype(np.float32)).to(out_kind)  # exact in fp32
        np.testing.assert_array_equal(whole[:, :cols].float().cpu().numpy(), want.float().numpy())


@pytest.mark.parametrize("block", [16, 32])
def test_quantize_what_is_not_finite(sampler, block):
    import torch

    x = torch.randn((200, 400), device="cuda:0")
    x[3, 5], x[150, 390], x[7, 130] = float("nan"), float("inf"), -float("inf")
    x[9] = float("nan")
    got, scales, row_scale = _quantize(sampler, x, block)
    codes, want_scales, want_row, values = M.quantize(x.cpu().numpy(), block)
    np.testing.assert_array_equal(row_scale.cpu().numpy(), want_row)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_scales)
    np.testing.assert_array_equal(got.cpu().numpy(), codes)
    back = torch.empty((200, 400), device="cuda:0")
    sampler.micro_rows(values=got, scales=scales, row_scale=row_scale, block=block, out=back)
    np.testing.assert_array_equal(back.cpu().numpy(), values.astype(np.float32))


@pytest.mark.parametrize("cols,kind", [(96, "bf16"), (333, "f32"), (4096, "bf16"), (257, "bf16")])
@pytest.mark.parametrize("block", [16, 32])
def test_rows_by_id(sampler, cols, kind, block):
    """An embedding's rows: ids in any order, twice, and outside."""
    import torch

    rng = np.random.default_rng(cols)
    t, _ = _source(rng, 300, cols, kind)
    got, scales, row_scale = _quantize(sampler, t.cuda(), block)
    row_scale = row_scale * 1.37  # a row scale of a user's own: products that round
    ids = torch.tensor([299, 0, 7, 7, -1, 300, 150, 2 ** 31 - 1, 128], dtype=torch.int32, device="cuda:0")
    out = torch.full((9, cols), -7.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda:0")
    sampler.micro_rows(values=got, scales=scales, row_scale=row_scale, ids=ids, block=block, out=out)
    want = M.values(got.cpu().numpy(), scales.cpu().numpy(), row_scale.cpu().numpy(), cols, block)
    out = out.double().cpu().numpy()
    half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -24
    for i, r in enumerate(ids.tolist()):
        if 0 <= r < 300:
            assert (np.abs(out[i] - want[r]) <= (half + 2 * 2.0 ** -24) * 1.01 * np.abs(want[r]) + 1e-45).all()
        else:
            assert np.isnan(out[i]).all()


@pytest.mark.parametrize("cols", [1, 7, 31, 33, 97, 500])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
def test_rows_to_anywhere(sampler, cols, kind, block):
    """Rows back to outputs that begin at each place of a vector, with guards around."""
    import torch

    rng = np.random.default_rng(cols)
    t, _ = _source(rng, 40, cols, "bf16")
    got, scales, row_scale = _quantize(sampler, t.cuda(), block)
    want = M.values(got.cpu().numpy(), scales.cpu().numpy(), row_scale.cpu().numpy(), cols, block)
    dtype = torch.bfloat16 if kind == "bf16" else torch.float32
    want = torch.from_numpy(want.astype(np.float32)).to(dtype).float().numpy()
    for shift in range(8):
        for gap in (0, 8 - cols % 8, 5):  # rows that begin one after the other, each at the same place, and elsewhere
            flat = torch.full((40 * (cols + gap) + shift + 40,), -7.0, dtype=dtype, device="cuda:0")
            view = flat[shift:shift + 40 * (cols + gap)].view(40, cols + gap)
            sampler.micro_rows(values=got, scales=scales, row_scale=row_scale, block=block, out=view[:, :cols])
            np.testing.assert_array_equal(view[:, :cols].float().cpu().numpy(), want)
            assert (view[:, cols:] == -7).all() and (flat[:shift] == -7).all() and (flat[-40:] == -7).all()


@pytest.mark.parametrize("cols,pad", [(64, 0), (128, 0), (33, 0), (256, 8), (1000, 0), (1024, 0), (1001, 1)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
def test_many_rows_are_as_few(sampler, cols, pad, kind, block):
    """So many rows that a thread has several in hand: the bytes of their first and last 1024 rows, quantised and read back
    apart."""
    import torch

    rows, few = 45003, 1024
    gen = torch.Generator(device="cuda:0").manual_seed(cols)
    whole = torch.randn((rows, cols + pad), generator=gen, device="cuda:0").to(torch.bfloat16 if kind == "bf16" else torch.float32)
    src = whole[:, :cols]
    values, scales, row_scale = _quantize(sampler, src, block)
    back = torch.full((rows, cols), -7.0, dtype=src.dtype, device="cuda:0")
    sampler.micro_rows(values=values, scales=scales, row_scale=row_scale, out=back, block=block)
    size = sampler.micro_scale_bytes(few, cols, block)
    start = (rows - few) // 128 * 128
    for at, n in ((0, few), (start, rows - start)):
        v, s, r = _quantize(sampler, src[at:at + n], block)
        assert torch.equal(values[at:at + n], v) and torch.equal(row_scale[at:at + n], r)
        first = at // 128 * (size // (few // 128))
        assert torch.equal(scales[first:first + s.numel()], s)
        out = torch.empty((n, cols), dtype=src.dtype, device="cuda:0")
        sampler.micro_rows(values=v, scales=s, row_scale=r, out=out, block=block)
        assert torch.equal(back[at:at + n], out)


def _operand(rng, rows, K, block, row_scale=True):
    """Random codes and scales: every code, scales of all sizes with zeros among them."""
    half = (K + 1) // 2
    packed = rng.integers(0, 256, (rows, half)).astype(np.uint8)
    if K % 2:
        packed[:, -1] &= 15
    place, size = M.scale_place(rows, K, block)
    scales = np.zeros(size, np.uint8)
    if block == 16:
        s = rng.integers(0x20, 0x60, place.shape)
        s[rng.random(place.shape) < 0.02] = 0
        s[rng.random(place.shape) < 0.02] = 0x7e
    else:
        s = rng.integers(117, 131, place.shape)
    scales[place] = s
    rs = (rng.uniform(0.001, 0.01, rows)).astype(np.float32) if row_scale else None
    return packed, scales, rs, M.values(packed, scales, rs, K, block)


def _up(packed, stride=None):
    """Codes on the device with rows `stride` apart; what lies between is 6."""
    import torch

    rows, half = packed.shape
    stride = stride or -(-half // 16) * 16
    t = torch.full((rows, stride), 0x77, dtype=torch.uint8, device="cuda:0")
    t[:, :half] = torch.from_numpy(packed).to("cuda:0")
    return t[:, :half]


def _dev(a):
    import torch

    return None if a is None else torch.from_numpy(a).to("cuda:0")


def _close(got, want, mag, K, kind):
    bound = (K * 2.0 ** -23 + 2 * 2.0 ** -24) * mag
    half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -24
    bad = ~(np.abs(got - want) <= half * np.abs(want) + (1 + half) * bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


SHAPES = [(1, 1, 1), (1, 128, 64), (2, 129, 65), (3, 1000, 32), (16, 4096, 256), (17, 300, 1000), (31, 5003, 96),
          (33, 640, 257), (64, 2000, 512), (65, 257, 129), (127, 640, 384), (128, 1024, 1024), (129, 1025, 300),
          (200, 3001, 256), (255, 511, 200), (256, 256, 4096), (257, 1300, 640), (513, 900, 16), (700, 1111, 1000),
          # few tiles with many stages of K
          (1, 1, 600), (16, 1000, 4096), (5, 4000, 2500), (40, 3000, 4100), (100, 500, 1900), (150, 130, 8200),
          # several tiles for each CTA, with more than one ring's stages
          (140, 42000, 1300), (300, 42001, 2100), (600, 20003, 384), (40, 40011, 2100), (128, 40000, 700),
          # tiles of two CTAs: few, several for each pair, a last one whose second CTA has no rows
          (256, 20000, 100), (511, 42001, 2100), (700, 30001, 64), (2600, 9003, 300)]


@pytest.mark.parametrize("rows,V,K", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
def test_product(sampler, rows, V, K, kind, block):
    import torch

    rng = np.random.default_rng(rows * 7 + V)
    h, sh, rh, hv = _operand(rng, rows, K, block)
    w, sw, rw, wv = _operand(rng, V, K, block, row_scale=V % 2 == 0)
    out = torch.full((rows, V + 3), -7.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda:0")
    sampler.lm_head_micro(hidden=_up(h), hidden_scale=_dev(sh), hidden_row_scale=_dev(rh),
                          weight=_up(w, -(-w.shape[1] // 16) * 16 + 32), weight_scale=_dev(sw), weight_row_scale=_dev(rw),
                          hidden_dim=K, block=block, logits=out)
    got = out.double().cpu().numpy()
    assert (got[:, V:] == -7).all(), "written beside the logits"
    want, mag = M.head(hv, wv)
    _close(got[:, :V], want, mag, K, kind)


@pytest.mark.parametrize("rows,V,K", [(200, 3000, 512), (300, 3008, 300), (129, 256, 64), (2600, 9008, 320)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_product_on_whole_vectors(sampler, rows, V, K, kind):
    """Logits that the TMA engine stores, with guards after the last row and beside."""
    import torch

    rng = np.random.default_rng(V)
    h, sh, rh, hv = _operand(rng, rows, K, 16)
    w, sw, rw, wv = _operand(rng, V, K, 16)
    out = torch.full((rows + 2, V + 16), -7.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda:0")
    sampler.lm_head_micro(hidden=_up(h), hidden_scale=_dev(sh), hidden_row_scale=_dev(rh), weight=_up(w),
                          weight_scale=_dev(sw), weight_row_scale=_dev(rw), hidden_dim=K, block=16, logits=out[:rows])
    got = out.double().cpu().numpy()
    assert (got[:, V:] == -7).all() and (got[rows:] == -7).all()
    want, mag = M.head(hv, wv)
    _close(got[:rows, :V], want, mag, K, kind)


@pytest.mark.parametrize("rows", [5, 200])
@pytest.mark.parametrize("block", [16, 32])
def test_what_is_not_finite_stays_in_its_rows(sampler, rows, block):
    """A block with a NaN makes its row's logits NaN, those of a hidden row or of a token, and no others."""
    import torch

    V, K = 700, 320
    gen = torch.Generator(device="cuda:0").manual_seed(3)
    hidden = torch.randn((rows, K), generator=gen, device="cuda:0")
    weight = torch.randn((V, K), generator=gen, device="cuda:0")
    hidden[2, 100], weight[300, 0], weight[699, 319] = float("nan"), float("inf"), float("nan")
    ops = {}
    for name, src in (("hidden", hidden), ("weight", weight)):
        ops[name], ops[name + "_scale"], ops[name + "_row_scale"] = _quantize(sampler, src, block)
    out = torch.empty((rows, V), device="cuda:0")
    sampler.lm_head_micro(**ops, hidden_dim=K, block=block, logits=out)
    want = torch.zeros((rows, V), dtype=torch.bool, device="cuda:0")
    want[2], want[:, 300], want[:, 699] = True, True, True
    assert torch.equal(torch.isnan(out), want) and torch.isfinite(out[~want]).all()


def _case(sampler, rows, V, K, block, seed=0):
    import torch

    rng = np.random.default_rng(seed)
    h, sh, rh, hv = _operand(rng, rows, K, block)
    w, sw, rw, wv = _operand(rng, V, K, block)
    return dict(hidden=_up(h), hidden_scale=_dev(sh), hidden_row_scale=_dev(rh), weight=_up(w), weight_scale=_dev(sw),
                weight_row_scale=_dev(rw), hidden_dim=K, block=block), hv, wv


@pytest.mark.parametrize("rows,K", [(24, 512), (150, 300)])
def test_stream_and_graph(sampler, rows, K):
    """On a stream of its own, captured with the quantiser before it, and replayed on other inputs: the same bits."""
    import torch

    V = 3000
    gen = torch.Generator(device="cuda:0").manual_seed(K)
    ops, _, _ = _case(sampler, rows, V, K, 16)
    hidden = torch.randn((rows, K), generator=gen, device="cuda:0").to(torch.bfloat16)
    values, scales, row_scale = _quantize(sampler, hidden, 16)
    ops |= dict(hidden=values, hidden_scale=scales, hidden_row_scale=row_scale)
    out = torch.empty((rows, V), device="cuda:0")

    def step():
        sampler.quantize_micro(src=hidden, out_values=values, out_scales=scales, out_row_scale=row_scale, block=16)
        sampler.lm_head_micro(**ops, logits=out)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    hidden.mul_(-0.5)  # a power of two: the same codes with the other sign, half the row scales
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -0.5 * first)


@pytest.mark.parametrize("rows", [1, 40, 256])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_chained_to_the_sampler(sampler, rows, kind):
    """The step after the head samples the head's logits."""
    import torch

    V, K = 5000, 640
    ops, _, _ = _case(sampler, rows, V, K, 32, seed=rows)
    dt = torch.bfloat16 if kind == "bf16" else torch.float32
    alone, chained = torch.empty((rows, V), dtype=dt, device="cuda:0"), torch.empty((rows, V), dtype=dt, device="cuda:0")
    sampler.lm_head_micro(**ops, logits=alone)
    temperature = torch.full((rows,), 0.8, device="cuda:0")
    tok, tok2 = (torch.empty(rows, dtype=torch.int32, device="cuda:0") for _ in range(2))
    lp, lp2 = torch.empty(rows, device="cuda:0"), torch.empty(rows, device="cuda:0")
    args = sampler.make_args(logits=alone, temperature=temperature, out_tokens=tok, global_seed=7)
    sampler.sample_ex_args(args, out_token_logprob=lp)
    args = sampler.make_args(logits=chained, temperature=temperature, out_tokens=tok2, global_seed=7)
    sampler.lm_head_micro_sample_args(args, out_token_logprob=lp2, **ops)
    assert torch.equal(alone, chained) and torch.equal(tok, tok2) and torch.equal(lp, lp2)


@pytest.mark.parametrize("rows", [40, 300])
def test_waits_that_give_up(rows):
    """With waits that give up at once the logits stay as they were and the blocks are counted; a handle after it works."""
    import torch

    import decode_step_token_gb300 as d

    with d.Sampler(max_rows=512, max_vocab=4096, short_waits=True) as s:
        ops, _, _ = _case(s, rows, 3000, 512, 16)
        out = torch.full((rows, 3000), -7.0, device="cuda:0")
        s.lm_head_micro(**ops, logits=out)
        assert s.stat(d.SAMPLER_STAT_LM_HEAD_TIMEOUTS) > 0
        assert (out == -7).all()
    with d.Sampler(max_rows=512, max_vocab=4096) as s:
        ops, hv, wv = _case(s, rows, 3000, 512, 16)
        s.lm_head_micro(**ops, logits=out)
        assert s.stat(d.SAMPLER_STAT_LM_HEAD_TIMEOUTS) == 0
        want, mag = M.head(hv, wv)
        _close(out.double().cpu().numpy(), want, mag, 512, "f32")


def _pair_case(sampler, block, nan=False):
    """So much that pairs of CTAs take it, of 300 rows by 20000 tokens."""
    import torch

    rows, V, K = 300, 20000, 2048
    gen = torch.Generator(device="cuda:0").manual_seed(block)
    hidden = torch.randn((rows, K), generator=gen, device="cuda:0")
    weight = torch.randn((V, K), generator=gen, device="cuda:0") / K ** 0.5
    if nan:
        hidden[2, 100], hidden[299, 2047], weight[300, 0], weight[19999, 319] = (float("nan"), float("inf"), float("-inf"),
                                                                               float("nan"))
    ops = dict(block=block)
    for name, src in (("hidden", hidden), ("weight", weight)):
        ops[name], ops[name + "_scale"], ops[name + "_row_scale"] = _quantize(sampler, src, block)
    return ops, torch.empty((rows, V), device="cuda:0")


@pytest.mark.parametrize("block", [16, 32])
def test_pairs_of_ctas_leave_nan_in_its_rows(sampler, block):
    import torch

    ops, out = _pair_case(sampler, block, nan=True)
    sampler.lm_head_micro(**ops, logits=out)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[[2, 299]], want[:, [300, 19999]] = True, True
    assert torch.equal(torch.isnan(out), want) and torch.isfinite(out[~want]).all()


def test_pairs_of_ctas_again_and_in_a_graph(sampler):
    """The same bits from every call, on two handles and streams at once, and from a graph, in which the sampler follows."""
    import torch

    import decode_step_token_gb300 as d

    ops, out = _pair_case(sampler, 16)
    sampler.lm_head_micro(**ops, logits=out)
    first = out.clone()
    with d.Sampler(max_rows=512, max_vocab=20000) as other:
        outs = [torch.empty_like(out) for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(5):
            for s, stream, to in zip((sampler, other), streams, outs):
                with torch.cuda.stream(stream):
                    s.lm_head_micro(**ops, logits=to)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    small = {k: v if k.startswith("weight") or k == "block" else v[:256] if k != "hidden_scale" else v for k, v in ops.items()}
    temperature = torch.full((256,), 0.8, device="cuda:0")
    tokens = torch.empty(256, dtype=torch.int32, device="cuda:0")
    args = sampler.make_args(logits=first[:256].contiguous(), temperature=temperature, out_tokens=tokens, global_seed=3)
    sampler.sample_ex_args(args)
    want = tokens.clone()
    chained = torch.empty((256, 20000), device="cuda:0")
    args = sampler.make_args(logits=chained, temperature=temperature, out_tokens=tokens, global_seed=3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sampler.lm_head_micro_sample_args(args, **small)
    for _ in range(3):
        tokens.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(chained, first[:256]) and torch.equal(tokens, want)


def test_pairs_of_ctas_whose_waits_give_up():
    import decode_step_token_gb300 as d

    with d.Sampler(max_rows=512, max_vocab=20000, short_waits=True) as s:
        ops, out = _pair_case(s, 16)
        out.fill_(-7.0)
        s.lm_head_micro(**ops, logits=out)
        assert s.stat(d.SAMPLER_STAT_LM_HEAD_TIMEOUTS) > 0 and (out == -7).all()


@pytest.mark.parametrize("rows", [5, 140])
def test_rows_far_apart(sampler, rows):
    """Offsets beyond 32 bits: of the source, the values, what is read back and the logits."""
    import torch

    V, K = 700, 320
    gen = torch.Generator(device="cuda:0").manual_seed(rows)
    hidden = torch.randn((rows, K), generator=gen, device="cuda:0").to(torch.bfloat16)
    weight = torch.randn((V, K), generator=gen, device="cuda:0").to(torch.bfloat16)

    def far(n, cols, dtype, apart):
        return torch.empty(n * apart, dtype=dtype, device="cuda:0").view(n, apart)[:, :cols]

    apart = 16 * (2 ** 32 // 16 // (rows - 1) + 1)  # in bytes, and more of what is larger
    src = far(rows, K, torch.bfloat16, apart)
    src.copy_(hidden)
    near = _quantize(sampler, hidden, 16)
    values = far(rows, K // 2, torch.uint8, apart)
    scales, row_scale = torch.empty_like(near[1]), torch.empty_like(near[2])
    sampler.quantize_micro(src=src, out_values=values, out_scales=scales, out_row_scale=row_scale)
    assert torch.equal(values, near[0]) and torch.equal(scales, near[1]) and torch.equal(row_scale, near[2])
    back, want = far(rows, K, torch.bfloat16, apart), torch.empty_like(hidden)
    sampler.micro_rows(values=near[0], scales=scales, row_scale=row_scale, out=want)
    sampler.micro_rows(values=values, scales=scales, row_scale=row_scale, out=back)
    assert torch.equal(back, want)
    w = _quantize(sampler, weight, 16)
    ops = dict(hidden_scale=scales, hidden_row_scale=row_scale, weight=w[0], weight_scale=w[1], weight_row_scale=w[2])
    logits, want = far(rows, V, torch.bfloat16, apart), torch.empty((rows, V), dtype=torch.bfloat16, device="cuda:0")
    sampler.lm_head_micro(hidden=near[0], logits=want, **ops)
    sampler.lm_head_micro(hidden=values, logits=logits, **ops)
    assert torch.equal(logits, want)


def test_argument_checks(sampler):
    import torch

    ops, _, _ = _case(sampler, 8, 300, 100, 16)
    out = torch.empty((8, 300), device="cuda:0")
    for change, error in [(dict(hidden=ops["hidden"].float()), TypeError), (dict(hidden_dim=98), ValueError),
                          (dict(hidden_scale=ops["hidden_scale"][:-1]), ValueError), (dict(block=24), ValueError),
                          (dict(weight_scale=ops["weight_scale"].float()), TypeError),
                          (dict(hidden_row_scale=ops["hidden_row_scale"][:7]), ValueError),
                          (dict(weight=ops["weight"].cpu()), ValueError), (dict(logits=out[:, :299]), ValueError)]:
        with pytest.raises(error):
            sampler.lm_head_micro(**{**dict(logits=out), **ops, **change})
    src = torch.randn((8, 100), device="cuda:0")
    q = dict(src=src, out_values=torch.empty((8, 50), dtype=torch.uint8, device="cuda:0"),
             out_scales=torch.empty(sampler.micro_scale_bytes(8, 100, 16), dtype=torch.uint8, device="cuda:0"),
             out_row_scale=torch.empty(8, device="cuda:0"))
    for change, error in [(dict(src=src.half()), TypeError), (dict(out_values=q["out_values"][:, :49]), ValueError),
                          (dict(out_scales=q["out_scales"][1:]), ValueError), (dict(block=8), ValueError),
                          (dict(out_row_scale=q["out_row_scale"][1:]), ValueError)]:
        with pytest.raises(error):
            sampler.quantize_micro(**{**q, **change})
    sampler.quantize_micro(**q)
    empty = torch.empty((0, 100), device="cuda:0")
    sampler.quantize_micro(src=empty, out_values=torch.empty((0, 50), dtype=torch.uint8, device="cuda:0"),
                           out_scales=q["out_scales"], out_row_scale=q["out_row_scale"])
    with pytest.raises(ValueError):
        sampler.micro_rows(values=q["out_values"], scales=q["out_scales"], out=torch.empty((8, 98), device="cuda:0"))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
def test_quantize_at_the_ends_of_the_types(sampler, block, kind):
    """The largest and the smallest values and scales, and largest values on the borders between two scales."""
    import torch

    rng = np.random.default_rng(block)
    cols, largest = 192, 3.3895314e38 if kind == "bf16" else 3.4028235e38
    up = np.float32(2.0 ** -7 if kind == "bf16" else 2.0 ** -23)
    x = np.zeros((140, cols), np.float32)
    x[0], x[1] = largest, -largest
    x[2] = (largest * rng.uniform(-1, 1, cols)).astype(np.float32)
    x[3], x[4] = 1.1754944e-38, 1e-45 if kind == "f32" else 9.2e-41  # least normal, least subnormal
    x[5] = (1e-38 * rng.standard_normal(cols)).astype(np.float32)
    x[6] = (1e-42 * rng.standard_normal(cols)).astype(np.float32)
    x[7] = np.where(rng.random(cols) < 0.5, 3e38, 1e-38)
    x[8] = np.where(np.arange(cols) < 64, largest, 1.0)
    x[9] = np.where(np.arange(cols) < 64, 2.0 ** -100, 2.0 ** -112)
    x[10] = 2.0 ** -100 * (1 + up)
    x[11, 5] = np.float32(2.0 ** -126)
    for r in range(12, 140):  # a largest value on a border of the scales, and one step on either side
        e = float(rng.integers(-120, 120))
        m = np.float32((1.3125 if r % 2 else 1.5) * 2.0 ** e) * (1 + up * np.float32(r % 3 - 1))
        x[r] = (float(m) * rng.choice([1.0, 0.5, 0.25, 0.125, 0.375, 0.625, 1 / 12], cols)).astype(np.float32)
        x[r, r] = m
    t = torch.from_numpy(x).to(torch.bfloat16 if kind == "bf16" else torch.float32)
    got, scales, row_scale = _quantize(sampler, t.to("cuda:0"), block)
    codes, want_scales, want_row, values = M.quantize(t.float().numpy(), block)
    np.testing.assert_array_equal(row_scale.cpu().numpy(), want_row)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_scales)
    np.testing.assert_array_equal(got.cpu().numpy(), codes)
    for out_kind in (torch.bfloat16, torch.float32):
        out = torch.empty((140, cols), dtype=out_kind, device="cuda:0")
        sampler.micro_rows(values=got, scales=scales, row_scale=row_scale, block=block, out=out)
        with np.errstate(over="ignore"):  # the largest may be rounded up to 2^128
            want = torch.from_numpy(values.astype(np.float32)).to(out_kind)
        np.testing.assert_array_equal(out.float().cpu().numpy(), want.float().numpy())


@pytest.mark.parametrize("rows", [9, 100, 300])
@pytest.mark.parametrize("far", [30, 60, 90])
@pytest.mark.parametrize("block", [16, 32])
def test_product_of_large_and_small_operands(sampler, rows, far, block):
    """Hidden rows of the size of 2^far by a weight of the size of 2^-far, and the other way round."""
    import torch

    V, K = 1300, 320
    rng = np.random.default_rng(far)
    for sign in (1, -1):
        hidden = (rng.standard_normal((rows, K)) * 2.0 ** (sign * far)).astype(np.float32)
        weight = (rng.standard_normal((V, K)) * 2.0 ** (-sign * far)).astype(np.float32)
        ops, exact = {}, {}
        for name, src in (("hidden", hidden), ("weight", weight)):
            ops[name], ops[name + "_scale"], ops[name + "_row_scale"] = _quantize(sampler, torch.from_numpy(src).cuda(), block)
            exact[name] = M.quantize(src, block)[3]
        out = torch.empty((rows, V), device="cuda:0")
        sampler.lm_head_micro(**ops, hidden_dim=K, block=block, logits=out)
        want, mag = M.head(exact["hidden"], exact["weight"])
        _close(out.double().cpu().numpy(), want, mag, K, "f32")


@pytest.mark.parametrize("rows,V,K,block,kind", [(64, 128000, 4096, 16, "bf16"), (1, 151936, 2048, 32, "bf16"),
                                                 (32, 32000, 4096, 32, "bf16"), (64, 32000, 4096, 16, "f32"),
                                                 (200, 50257, 768, 16, "bf16")])
def test_a_decode_step_of_full_size(sampler, rows, V, K, block, kind):
    """The chained step's logits, tokens and logprobs are those of the head and the sampler one after the other."""
    import torch

    gen = torch.Generator(device="cuda:0").manual_seed(V)
    ops = dict(block=block)
    for name, n, size in (("hidden", rows, 1.0), ("weight", V, K ** -0.5)):
        src = (size * torch.randn((n, K), generator=gen, device="cuda:0")).to(torch.bfloat16)
        ops[name], ops[name + "_scale"], ops[name + "_row_scale"] = _quantize(sampler, src, block)
    dt = torch.bfloat16 if kind == "bf16" else torch.float32
    temperature = torch.full((rows,), 0.7, device="cuda:0")
    got = []
    for chained in (False, True):
        logits = torch.full((rows, V), float("nan"), dtype=dt, device="cuda:0")
        token, lp = torch.empty(rows, dtype=torch.int32, device="cuda:0"), torch.empty(rows, device="cuda:0")
        args = sampler.make_args(logits=logits, temperature=temperature, out_tokens=token, global_seed=11,
                                 top_k=torch.full((rows,), 50, dtype=torch.int32, device="cuda:0"))
        if chained:
            sampler.lm_head_micro_sample_args(args, out_token_logprob=lp, **ops)
        else:
            sampler.lm_head_micro(**ops, logits=logits)
            sampler.sample_ex_args(args, out_token_logprob=lp)
        assert torch.isfinite(logits).all() and (token >= 0).all() and (token < V).all()
        got.append((logits, token, lp))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,V,K", [(65, 30001, 96), (90, 25000, 1000), (128, 19600, 1024), (100, 41003, 33), (128, 40000, 1025)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
def test_product_of_short_hidden_rows(sampler, rows, V, K, kind, block):
    """65 to 128 rows, which short hidden dimensions take as wide tiles."""
    test_product(sampler, rows, V, K, kind, block)
