"""Several handles in one process: what one of them does takes nothing from another. Needs a GB300."""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    from decode_step_token_gb300 import build
    build.build_library()
    import decode_step_token_gb300 as d
    return d


def _codes(rng, rows, K):
    import torch

    return torch.from_numpy(rng.integers(0, 0x70, (rows, K)).astype(np.uint8)).cuda()


def test_8bit_heads_of_two_threads(pkg):
    """A head of 16 rows needs less shared memory than one of 32: two threads that call them in turn, each with its
    handle and stream, do not refuse each other's launches."""
    import torch

    rng = np.random.default_rng(1)
    K, V, calls = 128, 300, 3000
    w, ws = _codes(rng, V, K), torch.ones((3, 1), device="cuda:0")
    failed, start = [], threading.Barrier(2)

    def work(rows):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            h, hs = ops[rows]
            with pkg.Sampler(max_rows=64, max_vocab=V) as s:
                start.wait()
                for _ in range(calls):
                    s.lm_head_scaled(hidden=h, hidden_scale=hs, weight=w, weight_scale=ws, logits=out[rows],
                                     stream=stream.cuda_stream)
                stream.synchronize()
        except Exception as e:  # noqa: BLE001 - seen by the test below
            failed.append((rows, e))

    ops = {rows: (_codes(rng, rows, K), torch.ones((rows, 1), device="cuda:0")) for rows in (16, 32)}
    out = {rows: torch.empty((rows, V), device="cuda:0") for rows in ops}
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(rows,)) for rows in ops]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_group_kernels_of_two_handles(pkg):
    """The fork-group kernel's shared memory follows the vocabulary: a small call of one handle leaves another's large
    one possible."""
    import torch

    def call(s, V, kind):
        x = torch.zeros((2, V), dtype=kind, device="cuda:0")
        x[:, 7] = 9.0
        tok = torch.empty(2, dtype=torch.int32, device="cuda:0")
        lp = torch.empty((2, V), device="cuda:0")
        s.sample(logits=x, temperature=torch.zeros(2, device="cuda:0"), out_tokens=tok, out_logprobs=lp)
        assert tok.tolist() == [7, 7]

    for kind in (torch.bfloat16, torch.float32):
        with pkg.Sampler(max_rows=4, max_vocab=262144) as a, pkg.Sampler(max_rows=4, max_vocab=262144) as b:
            call(a, 262144, kind)
            call(b, 100, kind)
            call(a, 262144, kind)


def test_lm_heads_of_two_handles(pkg):
    """So does the bf16 head's, with the rows."""
    import torch

    w = torch.eye(64, device="cuda:0").to(torch.bfloat16)

    def call(s, rows):
        h = w[torch.arange(rows, device="cuda:0") % 64]
        out = torch.empty((rows, 64), dtype=torch.bfloat16, device="cuda:0")
        s.lm_head(hidden=h, weight=w, logits=out)
        assert torch.equal(out, h)

    with pkg.Sampler(max_rows=256, max_vocab=64) as a, pkg.Sampler(max_rows=256, max_vocab=64) as b:
        sizes = (240, 16, 176, 256)
        for rows in sizes:
            call(a, rows)
        for rows in sizes[1:] + sizes:
            call(b, 16)
            call(a, rows)


def test_handle_for_any_number_of_rows(pkg):
    """max_rows only bounds the calls: a handle with a large one holds no memory for rows beyond what a loss takes."""
    import torch

    most = pkg.SAMPLER_LOSS_MAX_ROWS
    with pkg.Sampler(max_rows=1 << 40, max_vocab=1000) as s:
        x = torch.zeros((3, 1000), device="cuda:0")
        x[:, 5] = 60.0
        tok = torch.empty(3, dtype=torch.int32, device="cuda:0")
        s.sample(logits=x, temperature=torch.ones(3, device="cuda:0"), out_tokens=tok)
        assert tok.tolist() == [5, 5, 5]
        loss, one = torch.empty(1, device="cuda:0"), torch.ones(3, device="cuda:0")
        s.policy_loss(logits=x, tokens=tok, old_logprob=one - 1, advantage=one, out_loss=loss)
        assert abs(loss.item() + 3.0) < 1e-6
        # scoring takes more rows than the losses
        n = most + 5
        x = torch.zeros((n, 1), dtype=torch.bfloat16, device="cuda:0")
        tok, lp = torch.zeros(n, dtype=torch.int32, device="cuda:0"), torch.full((n,), -7.0, device="cuda:0")
        s.score(logits=x, tokens=tok, out_logprob=lp)
        assert (lp == 0).all()
        ends = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda:0")
        for call in (lambda: s.policy_loss(logits=x, tokens=tok, old_logprob=lp, advantage=lp, out_loss=loss),
                     lambda: s.preference_loss(logits=x, tokens=tok, seq_offsets=ends, out_loss=loss)):
            with pytest.raises(pkg.SamplerError) as e:
                call()
            assert e.value.code == -3
        s.policy_loss(logits=x[:most], tokens=tok, old_logprob=lp, advantage=lp, out_loss=loss)
        assert loss.item() == 0.0


def test_an_earlier_error_is_not_a_calls_own(pkg):
    """A handle that could not be had (its staging buffers are far larger than the memory) does not make the next
    calls of another report an error."""
    import torch

    x = torch.zeros((4, 256), device="cuda:0")
    codes, scales = torch.empty((4, 256), dtype=torch.float8_e4m3fn, device="cuda:0"), torch.empty((4, 2), device="cuda:0")
    tok, lp = torch.zeros(4, dtype=torch.int32, device="cuda:0"), torch.empty(4, device="cuda:0")
    with pkg.Sampler(max_rows=4, max_vocab=256) as s:
        for call in (lambda: s.score(logits=x, tokens=tok, out_logprob=lp),
                     lambda: s.quantize_blocks(src=x, out_values=codes, out_scales=scales)):
            with pytest.raises(pkg.SamplerError) as e:
                pkg.Sampler(max_rows=1 << 24, max_vocab=262144, host_staging=True)
            assert e.value.code == -5
            call()
    np.testing.assert_allclose(lp.cpu().numpy(), -np.log(256), rtol=1e-6)
