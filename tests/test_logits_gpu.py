"""Penalties, biases and masks on logits against an fp64 reference."""

import numpy as np
import pytest
import torch

from bit_weight_only_gemv_gb300 import lib
from oracle import serve

pytestmark = pytest.mark.gpu


def bits(t):
    return t.cpu().contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).numpy()


class Case:
    """B rows over V tokens; hist, nb: most tokens of a history and biases; masks: share allowed of
    each row or None."""

    def __init__(self, seed, B, V, hist=0, nb=0, masks=None, dtype=torch.bfloat16, pad=0, prompt=True,
                 penalties=True):
        rng = np.random.default_rng(seed)
        self.B, self.V, self.dtype = B, V, dtype
        full = torch.full((B, V + pad), 7.0, dtype=dtype, device="cuda")
        self.full = full
        self.logits = full[:, :V]
        self.logits.copy_(torch.from_numpy((rng.normal(size=(B, V)) * 4).astype(np.float32)))
        self.args = a = {}
        if hist:
            a["tokens"] = (V * rng.random((B, hist)) ** 3).astype(np.int32)
            a["lens"] = rng.integers(0, hist + 1, B).astype(np.int32)
            a["lens"][0] = hist
            if prompt:
                a["prompt"] = (a["lens"] * rng.random(B)).astype(np.int32)
        if penalties:
            a["repetition"] = (0.7 + rng.random(B)).astype(np.float32)
            a["presence"] = rng.normal(size=B).astype(np.float32)
            a["frequency"] = (rng.normal(size=B) * 0.2).astype(np.float32)
        if nb:
            a["bias_ids"] = rng.integers(0, V, (B, nb)).astype(np.int32)      # some of them twice
            a["bias"] = (rng.normal(size=(B, nb)) * 5).astype(np.float32)
            a["n_bias"] = rng.integers(0, nb + 1, B).astype(np.int32)
        self.allowed = [None] * B
        if masks is not None:
            rows = [b for b in range(B) if masks[b] is not None]
            words = -(-V // 32)
            m = np.zeros((max(1, len(rows)), words * 32), bool)
            for i, b in enumerate(rows):
                m[i] = rng.random(words * 32) < masks[b]
                self.allowed[b] = m[i, :V]
            packed = np.packbits(m.reshape(len(m), words, 32), axis=-1, bitorder="little")
            a["mask"] = np.ascontiguousarray(packed).view(np.int32).reshape(len(m), words)
            at = {b: i for i, b in enumerate(rows)}
            a["mask_rows"] = np.array([at.get(b, -1) for b in range(B)], np.int32)

    def rules(self, **over):
        return lib.LogitRules(**{k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v
                                 for k, v in {**self.args, **over}.items()})

    def check(self, left=(), code=None):
        """Rows in `left` keep their bits, and the call reports `code`.

        The repetition's reciprocal and its product, the frequency's fused product and difference, the
        presence's difference, the bias's sum: five roundings of 2^-24 of the terms' magnitudes at
        most, then half a step of the type."""
        a = self.args
        was, was_bits, around = self.logits.double().cpu().numpy(), bits(self.logits), bits(self.full)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lib.adjust_logits(self.logits, self.rules(), status)
        torch.cuda.synchronize()
        assert int(status) == (lib.STATUS_CODE[code] if code else 0)
        got, got_bits = self.logits.double().cpu().numpy(), bits(self.logits)
        assert np.array_equal(around[:, self.V:], bits(self.full)[:, self.V:])
        half = torch.finfo(self.dtype).eps / 2
        least = 5 * 2.0 ** -150 + (2.0 ** -134 if self.dtype == torch.bfloat16 else 0.0)
        for b in range(self.B):
            if b in left:
                assert np.array_equal(got_bits[b], was_bits[b])
                continue
            n = int(a["lens"][b]) if "lens" in a else 0
            nb = (int(a["n_bias"][b]) if "n_bias" in a else a["bias"].shape[1]) if "bias" in a else 0
            one = {k: float(a[k][b]) for k in ("repetition", "presence", "frequency") if k in a}
            ref, size, named = serve.adjust_row(
                was[b], a["tokens"][b, :n].tolist() if n else (),
                int(a["prompt"][b]) if "prompt" in a else 0, **one,
                bias=[(int(v), float(x)) for v, x in zip(a["bias_ids"][b, :nb], a["bias"][b, :nb])]
                if nb else (), mask=self.allowed[b])
            assert np.array_equal(got_bits[b][~named], was_bits[b][~named])
            with np.errstate(invalid="ignore"):
                # (below the smallest normal number a rounding is half the smallest number: 2^-150 of
                # 32 bits, 2^-134 of bf16)
                near = np.abs(got[b] - ref) <= 5 * 2.0 ** -24 * size + half * np.abs(ref) + least
            # beyond the type's largest number the result is infinite (or, by less than half a step,
            # that number)
            big = np.abs(ref) > torch.finfo(self.dtype).max
            near |= big & (got[b] == np.sign(ref) * np.inf)
            assert np.all(near | (got[b] == ref) | (np.isnan(ref) & np.isnan(got[b]))), b


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,V,hist,nb,masks,pad", [
    (1, 1, 3, 2, [0.5], 0), (2, 31, 5, 0, [None, 0.4], 0), (3, 1000, 0, 9, None, 0),
    (1, 262144, 700, 0, None, 0), (4, 8193, 300, 64, [None, 0.01, 0.99, 0.5], 5),
    (2, 20011, 5000, 4095, [0.3, None], 0), (3, 32768, 64, 3, [0.0, 1.0, 0.5], 8),
    (5, 50257, 2000, 20, None, 1), (2, 100277, 30000, 300, [0.05, 0.9], 0), (2, 64, 0, 0, [0.5, 0.0], 0)])
def test_rules(cuda_lib, dtype, B, V, hist, nb, masks, pad):
    Case(B + V, B, V, hist, nb, masks, dtype, pad).check()


@pytest.mark.parametrize("leave", ["prompt", "penalties", "repetition", "presence", "frequency", "n_bias",
                                   "all"])
def test_absent_rules(cuda_lib, leave):
    c = Case(5, 3, 4099, 200, 17, [0.5, None, 0.9])
    for k in {"penalties": ("repetition", "presence", "frequency"), "all": tuple(c.args)}.get(leave, (leave,)):
        del c.args[k]
    if leave == "all":
        c.allowed = [None] * 3
    c.check()


def test_a_mask_for_each_row_without_rows(cuda_lib):
    c = Case(6, 3, 5000, 10, 0, [0.2, 0.5, 0.8])
    del c.args["mask_rows"]
    c.check()


def test_rows_share_masks_and_strides(cuda_lib):
    """Histories, biases and masks as views of wider tensors; two rows under one mask."""
    c = Case(7, 3, 3001, 90, 12, [0.2, 0.5, None])
    c.args["mask_rows"] = np.array([1, 1, 0], np.int32)
    c.allowed = [c.allowed[1], c.allowed[1], c.allowed[0]]
    wide = {}
    for k in ("tokens", "bias_ids", "bias", "mask"):
        v = c.args[k]
        t = torch.full((v.shape[0], v.shape[1] + 7), -5, dtype=torch.from_numpy(v).dtype, device="cuda")
        t[:, :v.shape[1]] = torch.from_numpy(v).cuda()
        wide[k] = t[:, :v.shape[1]]
    rules = c.rules
    c.rules = lambda: rules(**wide)
    c.check()


def test_logits_that_are_not_finite(cuda_lib):
    c = Case(8, 2, 512, 400, 40, [0.5, None], torch.float32)
    c.logits[:, ::5] = float("inf")
    c.logits[:, 1::5] = float("-inf")
    c.logits[:, 2::5] = float("nan")
    c.check()
    c = Case(9, 1, 300, 50, 30)
    c.args["bias"][0, ::2] = -np.inf          # a ban
    c.args["bias"][0, 1::4] = np.inf
    c.check()


def test_one_token_many_times(cuda_lib):
    c = Case(10, 2, 9000, 40000, 0, None, torch.float32, prompt=False)
    c.args["tokens"][:] = 8999
    c.args["tokens"][1, ::2] = 3
    c.check()


@pytest.mark.parametrize("key,value,code", [
    ("lens", -1, "W4_ERR_INDEX"), ("lens", 201, "W4_ERR_INDEX"), ("prompt", -1, "W4_ERR_INDEX"),
    ("prompt", 201, "W4_ERR_INDEX"), ("n_bias", -1, "W4_ERR_INDEX"), ("n_bias", 18, "W4_ERR_INDEX"),
    ("mask_rows", -2, "W4_ERR_INDEX"), ("mask_rows", 3, "W4_ERR_INDEX"), ("repetition", 0, "W4_ERR_VALUE"),
    ("repetition", -1, "W4_ERR_VALUE"), ("repetition", np.nan, "W4_ERR_VALUE"),
    ("repetition", np.inf, "W4_ERR_VALUE"), ("presence", np.inf, "W4_ERR_VALUE"),
    ("frequency", np.nan, "W4_ERR_VALUE")])
def test_refused_rows_keep_their_bits(cuda_lib, key, value, code):
    c = Case(11, 4, 20000, 200, 17, [0.5, 0.9, 0.1, None])
    c.args[key][1] = value
    c.check(left=(1,), code=code)


@pytest.mark.parametrize("key", ["tokens", "bias_ids"])
@pytest.mark.parametrize("value", [-1, 20000, 2 ** 31 - 1, -2 ** 31])
def test_a_token_outside_the_vocabulary(cuda_lib, key, value):
    c = Case(12, 3, 20000, 200, 17, [0.5, 0.9, None])
    c.args["lens"][:] = 200
    c.args["n_bias"][:] = 17
    c.args[key][2, 9] = value
    c.check(left=(2,), code="W4_ERR_INDEX")
    c = Case(12, 3, 20000, 200, 17, [0.5, 0.9, None])       # past the counts: not read
    c.args["lens"][:] = 9
    c.args["prompt"][:] = 4
    c.args["n_bias"][:] = 9
    c.args[key][2, 9] = value
    c.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,V,hist,nb,masks,pad", [
    (16, 131075, 3, 2, [0.5, None, 0.999, 0.001], 0),          # a token or two named here and there
    (20, 262144, 9000, 40, [None, 0.97, 0.5, 0.02], 0),        # long histories, much work
    (90, 65536, 500, 10, [None, 0.9], 3), (700, 1000, 100, 3, [0.3, None], 0)])
def test_many_rows(cuda_lib, dtype, B, V, hist, nb, masks, pad):
    c = Case(B, B, V, hist, nb, [masks[b % len(masks)] for b in range(B)], dtype, pad)
    c.args["repetition"][3] = 1e-39            # a quotient that no reciprocal gives
    c.args["repetition"][4] = 3e38
    c.check()


@pytest.mark.parametrize("which", ["both", "tokens", "bias", "bias without counts", "slices"])
def test_lists_of_no_columns(cuda_lib, which):
    """No tokens yet, no biases in this batch: lists [rows, 0], which have no address of their own."""
    c = Case(13, 3, 4099, 8, 5, [0.5, None, 0.9])
    if which != "bias" and which != "bias without counts":
        c.args["tokens"] = c.args["tokens"][:, :0]
        c.args["lens"][:] = c.args["prompt"][:] = 0
    if which != "tokens":
        c.args["bias"], c.args["bias_ids"] = c.args["bias"][:, :0], c.args["bias_ids"][:, :0]
        c.args["n_bias"][:] = 0
    if which == "bias without counts":
        del c.args["n_bias"]
    if which == "slices":      # of tensors that are not empty
        rules, wide = c.rules, torch.full((3, 9), 7, dtype=torch.int32, device="cuda")
        c.rules = lambda: rules(tokens=wide[:, :0], bias_ids=wide[:, 3:3], bias=wide.float()[:, 2:2])
    c.check()


def test_counts_beyond_lists_of_no_columns(cuda_lib):
    c = Case(14, 4, 4099, 8, 5, [0.5, None, 0.9, None])
    c.args["tokens"] = c.args["tokens"][:, :0]
    c.args["bias"], c.args["bias_ids"] = c.args["bias"][:, :0], c.args["bias_ids"][:, :0]
    c.args["lens"][:] = c.args["prompt"][:] = c.args["n_bias"][:] = 0
    c.args["lens"][1] = c.args["n_bias"][3] = 1
    c.check(left=(1, 3), code="W4_ERR_INDEX")
