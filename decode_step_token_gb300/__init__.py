"""GB300-native per-decode-step token sampler, with what trains on its tokens.

The sampler itself is the CUDA library ``libsampler.so`` (C ABI in
``include/sampler.h``); this package is its thin Python binding. ``Sampler``
wraps a handle and takes torch tensors that already live on the GPU; PyTorch
provides device memory and streams only.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import _binding as abi
from ._binding import (EXPORTED, SAMPLER_CREATE_HOST_STAGING, SAMPLER_CREATE_SHORT_WAITS, SAMPLER_DTYPE_BF16,
                       SAMPLER_DTYPE_F32, SAMPLER_MAX_BIAS, SAMPLER_MAX_STOP, SAMPLER_MAX_TOP_N,
                       SAMPLER_LM_HEAD_MAX_ROWS, SAMPLER_NOALLOC_MAX_ROWS, SAMPLER_OK,
                       SAMPLER_STAT_EXACT_ROWS, SAMPLER_STAT_LM_HEAD_TIMEOUTS, sampler_lm_head_t,
                       sampler_lm_head_sample, sampler_lm_head,
                       load_library, sampler_abi_version, sampler_args_t, sampler_config_t, sampler_create,
                       sampler_destroy, sampler_ext_t, sampler_sample, sampler_sample_host,
                       sampler_sample_ex, sampler_sample_noalloc, sampler_status_string,
                       sampler_get_stat, SAMPLER_ERR_BAD_VALUE, SAMPLER_LOSS_MAX_ROWS, sampler_rows_t, sampler_policy_t,
                       sampler_preference_t, sampler_quantize_t, sampler_scaled_head_t, sampler_score,
                       sampler_score_grad, sampler_policy_loss, sampler_preference_loss, sampler_quantize_blocks,
                       sampler_lm_head_scaled, sampler_lm_head_scaled_sample, sampler_micro_t, sampler_micro_rows_t,
                       sampler_micro_head_t, sampler_micro_scale_bytes, sampler_quantize_micro, sampler_micro_rows,
                       sampler_lm_head_micro, sampler_lm_head_micro_sample, SAMPLER_MAX_ALTERNATIVES, sampler_top_t,
                       sampler_distill_t, sampler_score_top, sampler_distill_loss)

__all__ = ["Sampler", "SamplerError", "load_library", "sampler_create", "sampler_sample",
           "sampler_sample_host", "sampler_sample_noalloc", "sampler_sample_ex", "sampler_destroy",
           "sampler_status_string", "SAMPLER_NOALLOC_MAX_ROWS", "SAMPLER_MAX_TOP_N", "SAMPLER_MAX_BIAS",
           "SAMPLER_MAX_STOP", "sampler_ext_t", "sampler_lm_head_t", "sampler_lm_head_sample", "sampler_lm_head",
           "SAMPLER_LM_HEAD_MAX_ROWS", "SAMPLER_STAT_EXACT_ROWS", "SAMPLER_STAT_LM_HEAD_TIMEOUTS",
           "sampler_abi_version", "sampler_args_t", "sampler_config_t", "EXPORTED",
           "SAMPLER_ERR_BAD_VALUE", "SAMPLER_LOSS_MAX_ROWS", "sampler_rows_t", "sampler_policy_t", "sampler_preference_t",
           "sampler_quantize_t", "sampler_scaled_head_t", "sampler_score", "sampler_score_grad",
           "sampler_policy_loss", "sampler_preference_loss", "sampler_quantize_blocks", "sampler_lm_head_scaled",
           "sampler_lm_head_scaled_sample", "sampler_micro_t", "sampler_micro_rows_t", "sampler_micro_head_t",
           "sampler_micro_scale_bytes", "sampler_quantize_micro", "sampler_micro_rows", "sampler_lm_head_micro",
           "sampler_lm_head_micro_sample", "SAMPLER_MAX_ALTERNATIVES", "sampler_top_t", "sampler_distill_t",
           "sampler_score_top", "sampler_distill_loss"]


def _make_ext(top_n: int = 0, unscaled: bool = False, out_token_logprob=None, out_top_ids=None,
              out_top_logprobs=None, vocab_mask=None, mask_stride: Optional[int] = None, bias_offsets=None,
              bias_ids=None, bias_values=None, min_tokens_left=None, stop_offsets=None, stop_ids=None,
              sanitize_nan: bool = False) -> sampler_ext_t:
    if vocab_mask is not None and mask_stride is None:
        mask_stride = int(vocab_mask.shape[-1])
    return sampler_ext_t(int(top_n), 1 if unscaled else 0, _ptr(out_token_logprob), _ptr(out_top_ids),
                         _ptr(out_top_logprobs), _ptr(vocab_mask), int(mask_stride or 0),
                         _ptr(bias_offsets), _ptr(bias_ids), _ptr(bias_values),
                         _ptr(min_tokens_left), _ptr(stop_offsets), _ptr(stop_ids), 1 if sanitize_nan else 0)


class SamplerError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {sampler_status_string(code)} ({code})")
        self.code = code


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return int(t)


_raw_stream = None


def _current_stream(device: int) -> int:
    """The cudaStream_t of torch's current stream (its raw form where torch has one: a stream object costs microseconds)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream(device)  # torch's CUDA state is set up
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


_types = None


def _torch_types():
    """(bf16, fp32, int32, e4m3 and bytes) of torch, imported when it is first needed."""
    global _types
    if _types is None:
        import torch
        _types = (torch.bfloat16, torch.float32, torch.int32, (torch.float8_e4m3fn, torch.uint8))
    return _types


_micro = None


def _micro_types():
    """(those of two 4-bit values, those of their blocks' scales) of torch, as far as it has them, and bytes."""
    global _micro
    if _micro is None:
        import torch
        named = lambda *names: tuple(getattr(torch, n) for n in names if hasattr(torch, n))  # noqa: E731
        _micro = (named("uint8", "float4_e2m1fn_x2"), named("uint8", "float8_e4m3fn", "float8_e8m0fnu"))
    return _micro


def _scales(name: str, t, rows: int, cols: int, block: int, device: int) -> int:
    """Address of the scales of a matrix in 4 bits."""
    if block != 16 and block != 32:
        raise ValueError(f"{name}: no scales for blocks of {block} in {rows} x {cols}")
    # (sampler_micro_scale_bytes, without a call of the library, which checks the sizes itself)
    need = (rows + 127) // 128 * (((cols + block - 1) // block + 3) // 4) * 512
    if t.dtype in _micro_types()[1] and t.get_device() == device and t.numel() >= need and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in _micro_types()[1]:
        raise TypeError(f"{name} must be one of {_micro_types()[1]}, not {t.dtype}")
    _on_device(name, t, device)
    raise ValueError(f"{name} must be {need} contiguous bytes, not {tuple(t.shape)}")


def _vector(name: str, t, n: int, dtype, device: int) -> Optional[int]:
    """Address of a contiguous vector of n values or more on the handle's device (None passes)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == device and t.numel() >= n and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    _on_device(name, t, device)
    raise ValueError(f"{name} must be a contiguous vector of {n} values, not {tuple(t.shape)}")


def _matrix(name: str, t, dtypes, device: int):
    """(rows, columns, row stride) of a matrix on the handle's device with contiguous rows."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, not {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be two-dimensional with contiguous rows")
    rows, cols = t.shape
    stride, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must be two-dimensional with contiguous rows")
    if t.get_device() != device:
        _on_device(name, t, device)
    if stride < cols:
        if rows > 1:
            raise ValueError(f"{name}'s rows overlap: {stride} apart, {cols} wide")
        stride = cols
    return rows, cols, stride


def _on_device(name: str, t, device: int) -> None:
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")


class Sampler:
    """One libsampler handle on a CUDA device.

    ``sample`` takes device tensors: logits ``[rows, >= vocab]`` (bf16 or fp32, unit
    inner stride) and per-row parameter tensors, and writes the caller's output
    tensors. It enqueues on torch's current stream (or ``stream``) and returns
    without synchronising.
    """

    def __init__(self, max_rows: int, max_vocab: int, device: int = 0, max_history: int = 0,
                 host_staging: bool = False, short_waits: bool = False):
        flags = ((SAMPLER_CREATE_HOST_STAGING if host_staging else 0)
                 | (SAMPLER_CREATE_SHORT_WAITS if short_waits else 0))
        cfg = sampler_config_t(device, max_rows, max_vocab, max_history, flags)
        rc, h = sampler_create(cfg)
        if rc != SAMPLER_OK:
            raise SamplerError(rc, "sampler_create")
        self._h = h
        self.device = device
        self.max_rows = max_rows
        self.max_vocab = max_vocab

    def close(self):
        if getattr(self, "_h", None):
            sampler_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @staticmethod
    def make_args(*, logits, vocab=None, n_rows=None, temperature, dtype=None, top_k=None,
                  top_p=None, min_p=None, presence_penalty=None, frequency_penalty=None,
                  repetition_penalty=None, seed=None, has_seed=None, stream_id=None,
                  logit_row=None, hist_offsets=None, hist_ids=None, global_seed=0,
                  philox_offset=0, philox_offset_dev=None, out_tokens, out_probs=None,
                  out_logprobs=None, out_status=None, n_logit_rows=None,
                  row_stride=None) -> sampler_args_t:
        if dtype is None:
            import torch
            if logits.dtype == torch.bfloat16:
                dtype = SAMPLER_DTYPE_BF16
            elif logits.dtype == torch.float32:
                dtype = SAMPLER_DTYPE_F32
            else:
                raise TypeError(f"unsupported logits dtype {logits.dtype}")
        if row_stride is None:
            if logits.stride(-1) != 1:
                raise ValueError("logits rows must be contiguous")
            row_stride = logits.stride(0) if logits.dim() == 2 else logits.shape[-1]
        if vocab is None:
            vocab = logits.shape[-1]
        if n_rows is None:
            n_rows = temperature.shape[0]
        if n_logit_rows is None:
            n_logit_rows = logits.shape[0] if logits.dim() == 2 else 1
        return sampler_args_t(
            _ptr(logits), dtype, n_rows, vocab, row_stride, n_logit_rows, _ptr(logit_row),
            _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p), _ptr(presence_penalty),
            _ptr(frequency_penalty), _ptr(repetition_penalty), _ptr(seed), _ptr(has_seed),
            _ptr(stream_id), _ptr(hist_offsets), _ptr(hist_ids), global_seed, philox_offset,
            _ptr(philox_offset_dev), _ptr(out_tokens), _ptr(out_probs), _ptr(out_logprobs),
            _ptr(out_status))

    def sample_args(self, args: sampler_args_t, stream: Optional[int] = None) -> None:
        if stream is None:
            import torch
            stream = torch.cuda.current_stream(self.device).cuda_stream
        rc = sampler_sample(self._h, args, stream)
        if rc != SAMPLER_OK:
            raise SamplerError(rc, "sampler_sample")

    def sample(self, stream: Optional[int] = None, **kw) -> None:
        self.sample_args(self.make_args(**kw), stream)

    def sample_ex_args(self, args: sampler_args_t, top_n: int = 0, unscaled: bool = False,
                       out_token_logprob=None, out_top_ids=None, out_top_logprobs=None,
                       vocab_mask=None, mask_stride: Optional[int] = None,
                       bias_offsets=None, bias_ids=None, bias_values=None,
                       min_tokens_left=None, stop_offsets=None, stop_ids=None,
                       sanitize_nan: bool = False, stream: Optional[int] = None) -> None:
        """sampler_sample_ex: the step plus per-row logprob outputs (device tensors:
        out_token_logprob [N] fp32, out_top_ids / out_top_logprobs [N, top_n]
        int32 / fp32), a vocabulary bitmask (device [N, words] int32/uint32),
        logit_bias lists (device CSR: offsets [N + 1], ids, fp32 values), the
        min_tokens ban (device int32: tokens owed [N], stop-token CSR offsets
        [N + 1] and ids) and NaN sanitising."""
        ext = _make_ext(top_n, unscaled, out_token_logprob, out_top_ids, out_top_logprobs, vocab_mask,
                        mask_stride, bias_offsets, bias_ids, bias_values, min_tokens_left, stop_offsets,
                        stop_ids, sanitize_nan)
        rc = sampler_sample_ex(self._h, args, ext, self._stream(stream))
        if rc != SAMPLER_OK:
            raise SamplerError(rc, "sampler_sample_ex")

    def lm_head_sample_args(self, args: sampler_args_t, hidden, weight, hidden_dim: Optional[int] = None,
                            hidden_stride: Optional[int] = None, weight_stride: Optional[int] = None,
                            stream: Optional[int] = None, **ext_kw) -> None:
        """sampler_lm_head_sample: logits = hidden x weight^T (device bf16 tensors
        hidden [rows, K], weight [V, K]) written to args.logits, then the step on
        them; ext_kw as for sample_ex_args."""
        K = int(hidden_dim if hidden_dim is not None else hidden.shape[-1])
        lm = sampler_lm_head_t(_ptr(hidden), _ptr(weight), K,
                               int(hidden_stride if hidden_stride is not None else hidden.stride(0)),
                               int(weight_stride if weight_stride is not None else weight.stride(0)))
        ext = _make_ext(**ext_kw) if ext_kw else None
        rc = sampler_lm_head_sample(self._h, lm, args, ext, self._stream(stream))
        if rc != SAMPLER_OK:
            raise SamplerError(rc, "sampler_lm_head_sample")

    def lm_head(self, hidden, weight, logits, rows: Optional[int] = None, vocab: Optional[int] = None,
                hidden_dim: Optional[int] = None, hidden_stride: Optional[int] = None,
                weight_stride: Optional[int] = None, logits_stride: Optional[int] = None,
                stream: Optional[int] = None) -> None:
        """sampler_lm_head: logits = hidden x weight^T (device bf16 tensors hidden
        [rows, K], weight [V, K], logits [rows, stride])."""
        K = int(hidden_dim if hidden_dim is not None else hidden.shape[-1])
        lm = sampler_lm_head_t(_ptr(hidden), _ptr(weight), K,
                               int(hidden_stride if hidden_stride is not None else hidden.stride(0)),
                               int(weight_stride if weight_stride is not None else weight.stride(0)))
        rc = sampler_lm_head(self._h, lm, _ptr(logits),
                             int(logits_stride if logits_stride is not None else logits.stride(0)),
                             int(rows if rows is not None else hidden.shape[0]),
                             int(vocab if vocab is not None else weight.shape[0]), self._stream(stream))
        if rc != SAMPLER_OK:
            raise SamplerError(rc, "sampler_lm_head")

    def _rows(self, logits, tokens, temperature, weight, out_logprob, out_entropy, out_status, out_grad,
              vocab: Optional[int]) -> sampler_rows_t:
        bf16, f32, i32, _ = _torch_types()
        dev = self.device
        n, cols, stride = _matrix("logits", logits, (bf16, f32), dev)
        V = cols if vocab is None else int(vocab)
        if not 1 <= V <= cols:
            raise ValueError(f"vocab {V} does not lie within the logits' {cols} columns")
        grad, grad_stride = None, 0
        if out_grad is not None:
            gn, gcols, grad_stride = _matrix("out_grad", out_grad, (logits.dtype,), dev)
            if gn != n or gcols < V:
                raise ValueError(f"out_grad must be [{n}, {V}], not {tuple(out_grad.shape)}")
            grad = out_grad.data_ptr()
        return sampler_rows_t(
            logits.data_ptr(), SAMPLER_DTYPE_BF16 if logits.dtype is bf16 else SAMPLER_DTYPE_F32, n, V, stride,
            _vector("tokens", tokens, n, i32, dev), _vector("temperature", temperature, n, f32, dev),
            _vector("weight", weight, n, f32, dev), _vector("out_logprob", out_logprob, n, f32, dev),
            _vector("out_entropy", out_entropy, n, f32, dev), _vector("out_status", out_status, n, i32, dev), grad,
            grad_stride)

    def _done(self, rc: int, what: str) -> None:
        if rc != SAMPLER_OK:
            raise SamplerError(rc, what)

    def score(self, *, logits, tokens, out_logprob=None, out_entropy=None, out_status=None, temperature=None,
              weight=None, vocab: Optional[int] = None, stream: Optional[int] = None) -> None:
        """sampler_score: the logprob and the entropy of each row's token (int32
        tokens [N]; fp32 temperature, weight and outputs [N]; a row of weight 0 is
        left out)."""
        rows = self._rows(logits, tokens, temperature, weight, out_logprob, out_entropy, out_status, None, vocab)
        self._done(sampler_score(self._h, rows, self._stream(stream)), "sampler_score")

    def score_grad(self, *, logits, tokens, grad_logprob, out_grad, grad_entropy=None, out_logprob=None,
                   out_entropy=None, out_status=None, temperature=None, weight=None, vocab: Optional[int] = None,
                   stream: Optional[int] = None) -> None:
        """sampler_score_grad: the logits' gradient of sum(grad_logprob * logprob +
        grad_entropy * entropy) into out_grad (the logits' type; it may be the logits),
        with the outputs of ``score``."""
        rows = self._rows(logits, tokens, temperature, weight, out_logprob, out_entropy, out_status, out_grad, vocab)
        n, f32 = rows.n_rows, _torch_types()[1]
        gl = _vector("grad_logprob", grad_logprob, n, f32, self.device)
        ge = _vector("grad_entropy", grad_entropy, n, f32, self.device)
        self._done(sampler_score_grad(self._h, rows, gl, ge, self._stream(stream)), "sampler_score_grad")

    def score_top(self, *, logits, top_n: int, out_top_ids, out_top_logprobs, out_rest_logprob=None, tokens=None,
                  out_logprob=None, out_entropy=None, out_status=None, temperature=None, weight=None,
                  vocab: Optional[int] = None, stream: Optional[int] = None) -> None:
        """sampler_score_top: the top_n most likely tokens of each row (int32 out_top_ids,
        fp32 out_top_logprobs, [N, top_n]) and the logprob of all others together
        (fp32 out_rest_logprob [N]), with the outputs of ``score`` for tokens, where
        they are given."""
        rows = self._rows(logits, tokens, temperature, weight, out_logprob, out_entropy, out_status, None, vocab)
        n, (_, f32, i32, _), dev = rows.n_rows, _torch_types(), self.device
        q = sampler_top_t(top_n, _vector("out_top_ids", out_top_ids, n * max(0, top_n), i32, dev),
                          _vector("out_top_logprobs", out_top_logprobs, n * max(0, top_n), f32, dev),
                          _vector("out_rest_logprob", out_rest_logprob, n, f32, dev))
        self._done(sampler_score_top(self._h, rows, q, self._stream(stream)), "sampler_score_top")

    def distill_loss(self, *, logits, teacher_ids, teacher_logprobs, out_loss, teacher_rest=None, tokens=None,
                     token_coef: float = 0.0, temperature=None, weight=None, grad_scale: float = 1.0,
                     grad_scale_dev=None, out_grad=None, out_kl=None, out_logprob=None, out_status=None,
                     vocab: Optional[int] = None, stream: Optional[int] = None) -> None:
        """sampler_distill_loss against the lists that ``score_top`` gives of a teacher's
        rows (int32 teacher_ids and fp32 teacher_logprobs [N, n], fp32 teacher_rest
        [N]), with token_coef times the loss of tokens (out_loss: one fp32), and with
        out_grad the logits' gradient."""
        rows = self._rows(logits, tokens, temperature, weight, out_logprob, None, out_status, out_grad, vocab)
        n, (_, f32, i32, _), dev = rows.n_rows, _torch_types(), self.device
        if teacher_ids.dim() != 2 or teacher_ids.shape != teacher_logprobs.shape or teacher_ids.shape[0] != n:
            raise ValueError(f"teacher_ids and teacher_logprobs must be [{n}, top_n], not {tuple(teacher_ids.shape)} and "
                             f"{tuple(teacher_logprobs.shape)}")
        top_n = teacher_ids.shape[1]
        q = sampler_distill_t(top_n, _vector("teacher_ids", teacher_ids, n * top_n, i32, dev),
                              _vector("teacher_logprobs", teacher_logprobs, n * top_n, f32, dev),
                              _vector("teacher_rest", teacher_rest, n, f32, dev), token_coef, grad_scale,
                              _vector("grad_scale_dev", grad_scale_dev, 1, f32, dev),
                              _vector("out_loss", out_loss, 1, f32, dev), _vector("out_kl", out_kl, n, f32, dev))
        self._done(sampler_distill_loss(self._h, rows, q, self._stream(stream)), "sampler_distill_loss")

    def policy_loss(self, *, logits, tokens, old_logprob, advantage, out_loss, ref_logprob=None, temperature=None,
                    weight=None, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                    entropy_coef: float = 0.0, grad_scale: float = 1.0, grad_scale_dev=None, out_grad=None,
                    out_logprob=None, out_ratio=None, out_kl=None, out_entropy=None, out_status=None,
                    vocab: Optional[int] = None, stream: Optional[int] = None) -> None:
        """sampler_policy_loss: the clipped policy loss with its KL and entropy terms
        (out_loss: one fp32), and with out_grad the logits' gradient in the same pass."""
        rows = self._rows(logits, tokens, temperature, weight, out_logprob, out_entropy, out_status, out_grad, vocab)

        n, f32, dev = rows.n_rows, _torch_types()[1], self.device
        q = sampler_policy_t(_vector("old_logprob", old_logprob, n, f32, dev), _vector("advantage", advantage, n, f32, dev),
                             _vector("ref_logprob", ref_logprob, n, f32, dev), clip_low, clip_high, kl_coef,
                             entropy_coef, grad_scale, _vector("grad_scale_dev", grad_scale_dev, 1, f32, dev),
                             _vector("out_loss", out_loss, 1, f32, dev), _vector("out_ratio", out_ratio, n, f32, dev),
                             _vector("out_kl", out_kl, n, f32, dev))
        self._done(sampler_policy_loss(self._h, rows, q, self._stream(stream)), "sampler_policy_loss")

    def preference_loss(self, *, logits, tokens, seq_offsets, out_loss, ref_logprob=None, temperature=None,
                        weight=None, beta: float = 0.1, margin: float = 0.0, label_smoothing: float = 0.0,
                        mean_over_tokens: bool = False, grad_scale: float = 1.0, grad_scale_dev=None, out_grad=None,
                        out_logprob=None, out_reward=None, out_status=None, vocab: Optional[int] = None,
                        stream: Optional[int] = None) -> None:
        """sampler_preference_loss over (len(seq_offsets) - 1) / 2 pairs of answers
        (int32 seq_offsets; out_loss: one fp32; out_reward: one for each answer), and
        with out_grad the logits' gradient."""
        rows = self._rows(logits, tokens, temperature, weight, out_logprob, None, out_status, out_grad, vocab)
        ends = int(seq_offsets.shape[0])
        if ends % 2 != 1:
            raise ValueError(f"seq_offsets must have 2 * pairs + 1 entries, not {ends}")
        n, (_, f32, i32, _) = rows.n_rows, _torch_types()
        q = sampler_preference_t(_vector("seq_offsets", seq_offsets, ends, i32, self.device), ends // 2,
                                 _vector("ref_logprob", ref_logprob, n, f32, self.device), beta, margin,
                                 label_smoothing, 1 if mean_over_tokens else 0, grad_scale,
                                 _vector("grad_scale_dev", grad_scale_dev, 1, f32, self.device),
                                 _vector("out_loss", out_loss, 1, f32, self.device),
                                 _vector("out_reward", out_reward, ends - 1, f32, self.device))
        self._done(sampler_preference_loss(self._h, rows, q, self._stream(stream)), "sampler_preference_loss")

    def quantize_blocks(self, *, src, out_values, out_scales, block_rows: int = 1,
                        stream: Optional[int] = None) -> None:
        """sampler_quantize_blocks: src [rows, cols] (bf16 or fp32) to out_values
        (float8_e4m3fn, the same shape) with out_scales (fp32, [rows / block_rows,
        cols / 128] rounded up)."""
        bf16, f32, _, eight = _torch_types()
        rows, cols, stride = _matrix("src", src, (bf16, f32), self.device)
        vr, vc, vs = _matrix("out_values", out_values, eight, self.device)
        sr, sc, ss = _matrix("out_scales", out_scales, (f32,), self.device)
        if vr != rows or vc != cols:
            raise ValueError(f"out_values must be [{rows}, {cols}], not {tuple(out_values.shape)}")
        if block_rows > 0 and (sr < -(-rows // block_rows) or sc < -(-cols // 128)):
            raise ValueError(f"out_scales {tuple(out_scales.shape)} is too small for {rows} x {cols}")
        q = sampler_quantize_t(src.data_ptr(), SAMPLER_DTYPE_BF16 if src.dtype is bf16 else SAMPLER_DTYPE_F32, rows,
                               cols, stride, int(block_rows), out_values.data_ptr(), vs, out_scales.data_ptr(), ss)
        self._done(sampler_quantize_blocks(self._h, q, self._stream(stream)), "sampler_quantize_blocks")

    def _scaled_head(self, hidden, hidden_scale, weight, weight_scale) -> sampler_scaled_head_t:
        _, f32, _, eight = _torch_types()
        rows, K, hs = _matrix("hidden", hidden, eight, self.device)
        V, wk, ws = _matrix("weight", weight, eight, self.device)
        if wk != K:
            raise ValueError(f"hidden has {K} columns, weight {wk}")
        hr, hc, hss = _matrix("hidden_scale", hidden_scale, (f32,), self.device)
        wr, wc, wss = _matrix("weight_scale", weight_scale, (f32,), self.device)
        groups = -(-K // 128)
        if hr < rows or hc < groups:
            raise ValueError(f"hidden_scale must be [{rows}, {groups}], not {tuple(hidden_scale.shape)}")
        if wr < -(-V // 128) or wc < groups:
            raise ValueError(f"weight_scale must be [{-(-V // 128)}, {groups}], not {tuple(weight_scale.shape)}")
        # the stride of a single row is not used, but has to be a legal one
        if rows <= 1:
            hs = -(-hs // 16) * 16
        if V <= 1:
            ws = -(-ws // 16) * 16
        return sampler_scaled_head_t(hidden.data_ptr(), hidden_scale.data_ptr(), weight.data_ptr(),
                                     weight_scale.data_ptr(), K, hs, ws, hss, wss)

    def lm_head_scaled(self, *, hidden, hidden_scale, weight, weight_scale, logits,
                       stream: Optional[int] = None) -> None:
        """sampler_lm_head_scaled: logits [rows, >= vocab] (bf16 or fp32) from e4m3
        hidden [rows, K] and weight [vocab, K] with their scales as
        ``quantize_blocks`` makes them (block_rows 1 and 128)."""
        lm = self._scaled_head(hidden, hidden_scale, weight, weight_scale)
        bf16, f32, _, _ = _torch_types()
        lr, lc, ldl = _matrix("logits", logits, (bf16, f32), self.device)
        rows, V = hidden.shape[0], weight.shape[0]
        if lr < rows or lc < V:
            raise ValueError(f"logits must be [{rows}, {V}], not {tuple(logits.shape)}")
        dtype = SAMPLER_DTYPE_BF16 if logits.dtype is bf16 else SAMPLER_DTYPE_F32
        self._done(sampler_lm_head_scaled(self._h, lm, logits.data_ptr(), dtype, ldl, rows, V, self._stream(stream)),
                   "sampler_lm_head_scaled")

    def lm_head_scaled_sample_args(self, args: sampler_args_t, *, hidden, hidden_scale, weight, weight_scale,
                                   stream: Optional[int] = None, **ext_kw) -> None:
        """sampler_lm_head_scaled_sample: the logits of ``lm_head_scaled`` written to
        args.logits, then the step on them; ext_kw as for sample_ex_args."""
        lm = self._scaled_head(hidden, hidden_scale, weight, weight_scale)
        rows = args.n_logit_rows if args.n_logit_rows > 0 else args.n_rows
        if hidden.shape[0] < rows or weight.shape[0] < args.vocab:
            raise ValueError(f"hidden and weight must have {rows} and {args.vocab} rows")
        ext = _make_ext(**ext_kw) if ext_kw else None
        self._done(sampler_lm_head_scaled_sample(self._h, lm, args, ext, self._stream(stream)),
                   "sampler_lm_head_scaled_sample")

    @staticmethod
    def micro_scale_bytes(rows: int, cols: int, block: int = 16) -> int:
        """Bytes of the scales of a [rows, cols] matrix in 4 bits."""
        n = sampler_micro_scale_bytes(rows, cols, block)
        if n < 0:
            raise ValueError(f"no scales for blocks of {block} in {rows} x {cols}")
        return n

    def quantize_micro(self, *, src, out_values, out_scales, out_row_scale, block: int = 16,
                       stream: Optional[int] = None) -> None:
        """sampler_quantize_micro: src [rows, cols] (bf16 or fp32) to out_values (bytes
        of two 4-bit values, [rows, cols / 2] rounded up) with out_scales
        (``micro_scale_bytes``) and out_row_scale (fp32 [rows])."""
        bf16, f32, _, _ = _torch_types()
        dev = self.device
        rows, cols, stride = _matrix("src", src, (bf16, f32), dev)
        vr, vc, vs = _matrix("out_values", out_values, _micro_types()[0], dev)
        if vr != rows or vc != (cols + 1) // 2:
            raise ValueError(f"out_values must be [{rows}, {(cols + 1) // 2}], not {tuple(out_values.shape)}")
        q = sampler_micro_t(src.data_ptr(), SAMPLER_DTYPE_BF16 if src.dtype is bf16 else SAMPLER_DTYPE_F32, rows, cols,
                            stride, block, out_values.data_ptr(), vs,
                            _scales("out_scales", out_scales, rows, cols, block, dev),
                            _vector("out_row_scale", out_row_scale, rows, f32, dev))
        self._done(sampler_quantize_micro(self._h, q, self._stream(stream)), "sampler_quantize_micro")

    def micro_rows(self, *, values, scales, out, row_scale=None, ids=None, block: int = 16,
                   stream: Optional[int] = None) -> None:
        """sampler_micro_rows: rows of a matrix that ``quantize_micro`` has laid out back
        into out [n, cols] (bf16 or fp32): the rows that ids (int32 [n]) names, or the
        first n."""
        bf16, f32, i32, _ = _torch_types()
        dev = self.device
        rows, vc, vs = _matrix("values", values, _micro_types()[0], dev)
        n, cols, stride = _matrix("out", out, (bf16, f32), dev)
        if vc != (cols + 1) // 2:
            raise ValueError(f"out has {cols} columns, values has bytes for {2 * vc}")
        q = sampler_micro_rows_t(values.data_ptr(), vs, _scales("scales", scales, rows, cols, block, dev),
                                 _vector("row_scale", row_scale, rows, f32, dev), rows, cols, block,
                                 _vector("ids", ids, n, i32, dev), n, out.data_ptr(),
                                 SAMPLER_DTYPE_BF16 if out.dtype is bf16 else SAMPLER_DTYPE_F32, stride)
        self._done(sampler_micro_rows(self._h, q, self._stream(stream)), "sampler_micro_rows")

    def _micro_head(self, hidden, hidden_scale, weight, weight_scale, hidden_dim, hidden_row_scale, weight_row_scale,
                    block) -> sampler_micro_head_t:
        dev, f32, four = self.device, _torch_types()[1], _micro_types()[0]
        rows, hb, hs = _matrix("hidden", hidden, four, dev)
        V, wb, ws = _matrix("weight", weight, four, dev)
        K = 2 * hb if hidden_dim is None else int(hidden_dim)
        if hb != (K + 1) // 2 or wb != (K + 1) // 2:
            raise ValueError(f"hidden and weight must have {(K + 1) // 2} bytes a row, not {hb} and {wb}")
        # the stride of a single row is not used, but has to be a legal one
        if rows <= 1:
            hs = -(-hs // 16) * 16
        if V <= 1:
            ws = -(-ws // 16) * 16
        return sampler_micro_head_t(hidden.data_ptr(), _scales("hidden_scale", hidden_scale, rows, K, block, dev),
                                    _vector("hidden_row_scale", hidden_row_scale, rows, f32, dev), weight.data_ptr(),
                                    _scales("weight_scale", weight_scale, V, K, block, dev),
                                    _vector("weight_row_scale", weight_row_scale, V, f32, dev), K, hs, ws, block)

    def lm_head_micro(self, *, hidden, hidden_scale, weight, weight_scale, logits, hidden_dim: Optional[int] = None,
                      hidden_row_scale=None, weight_row_scale=None, block: int = 16,
                      stream: Optional[int] = None) -> None:
        """sampler_lm_head_micro: logits [rows, >= vocab] (bf16 or fp32) from hidden [rows,
        K / 2] and weight [vocab, K / 2] in 4 bits with their scales, as
        ``quantize_micro`` makes them. hidden_dim: K, where it is odd."""
        lm = self._micro_head(hidden, hidden_scale, weight, weight_scale, hidden_dim, hidden_row_scale, weight_row_scale,
                              block)
        bf16, f32, _, _ = _torch_types()
        lr, lc, ldl = _matrix("logits", logits, (bf16, f32), self.device)
        rows, V = hidden.shape[0], weight.shape[0]
        if lr < rows or lc < V:
            raise ValueError(f"logits must be [{rows}, {V}], not {tuple(logits.shape)}")
        dtype = SAMPLER_DTYPE_BF16 if logits.dtype is bf16 else SAMPLER_DTYPE_F32
        self._done(sampler_lm_head_micro(self._h, lm, logits.data_ptr(), dtype, ldl, rows, V, self._stream(stream)),
                   "sampler_lm_head_micro")

    def lm_head_micro_sample_args(self, args: sampler_args_t, *, hidden, hidden_scale, weight, weight_scale,
                                  hidden_dim: Optional[int] = None, hidden_row_scale=None, weight_row_scale=None,
                                  block: int = 16, stream: Optional[int] = None, **ext_kw) -> None:
        """sampler_lm_head_micro_sample: the logits of ``lm_head_micro`` written to
        args.logits, then the step on them; ext_kw as for sample_ex_args."""
        lm = self._micro_head(hidden, hidden_scale, weight, weight_scale, hidden_dim, hidden_row_scale, weight_row_scale,
                              block)
        rows = args.n_logit_rows if args.n_logit_rows > 0 else args.n_rows
        if hidden.shape[0] < rows or weight.shape[0] < args.vocab:
            raise ValueError(f"hidden and weight must have {rows} and {args.vocab} rows")
        ext = _make_ext(**ext_kw) if ext_kw else None
        self._done(sampler_lm_head_micro_sample(self._h, lm, args, ext, self._stream(stream)),
                   "sampler_lm_head_micro_sample")

    def _stream(self, stream: Optional[int]) -> int:
        return _current_stream(self.device) if stream is None else stream

    def stat(self, which: int = 0, reset: bool = False) -> int:
        """A device diagnostic counter (synchronizes the device)."""
        rc, v = sampler_get_stat(self._h, which, reset)
        if rc != SAMPLER_OK:
            raise SamplerError(rc, "sampler_get_stat")
        return v

    def sample_host_args(self, args: sampler_args_t, stream: int = 0) -> None:
        rc = sampler_sample_host(self._h, args, stream)
        if rc != SAMPLER_OK:
            raise SamplerError(rc, "sampler_sample_host")
