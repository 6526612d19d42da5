"""The attention-side operators without a GPU: the header's entry points are exported, argument errors are answered on
the host before any device work, and the index arithmetic of the attention tiles holds (compiled for the host)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import bit_quantized_linear_svdq_b200 as S
from bit_quantized_linear_svdq_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    B.build()
    return S.load_library()


def test_header_entry_points_are_exported(lib):
    with open(os.path.join(ROOT, "include", "svdq_attn.h")) as f:
        names = set(re.findall(r"SVDQ_API\s+[\w\s\*]+?\b(svdq_\w+)\s*\(", f.read()))
    assert names == {"svdq_qk_norm_rope", "svdq_kv4_append", "svdq_kv4_read", "svdq_kv4_attention_workspace_bytes",
                     "svdq_kv4_attention", "svdq_kv4_attention_status"}
    for n in names:
        assert hasattr(lib, n) and callable(getattr(S, n))


def test_structures_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = ["svdq_heads", "svdq_qk_norm_rope_desc", "svdq_kv4_cache", "svdq_kv4_attention_desc"]
    body = "".join(f'printf("%zu\\n", sizeof({n}));' for n in names)
    for n in names:
        body += "".join(f'printf("%zu\\n", offsetof({n}, {f}));' for f, *_ in getattr(S, n)._fields_)
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "svdq_attn.h"\nint main(void) {' + body + "return 0;}")
    exe = str(tmp_path / "sizes")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    want = [ctypes.sizeof(getattr(S, n)) for n in names]
    for n in names:
        want += [getattr(getattr(S, n), f).offset for f, *_ in getattr(S, n)._fields_]
    assert got == want


def test_rows_and_keys_of_the_tiles(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "kv4_rows_check")
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", B.CSRC, os.path.join(ROOT, "tests", "native", "kv4_rows_check.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert r.stdout.strip() == "ok"


# ------------------------------------------------------------------ C entry points: host-side errors

H = lambda ptr=256, ts=512, hs=128: S.svdq_heads(ptr, ts, hs)  # noqa: E731


def _rope(**kw):
    base = dict(tokens=4, q_heads=4, k_heads=2, head_dim=128, dtype=0, q=H(), k=H(), q_out=H(), k_out=H(), eps=1e-6,
                positions=256, position_stride=1, axes=1, inv_freq=256, pairs=64)
    base.update(kw)
    return S.svdq_qk_norm_rope_desc(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), 1), (dict(dtype=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(head_dim=4), 2), (dict(head_dim=264), 2), (dict(head_dim=100), 2),
    (dict(head_dim=96, hadamard=1, pairs=48), 2), (dict(q_heads=-1), 2), (dict(k_heads=70000), 2),
    (dict(pairs=-1), 2), (dict(pairs=72, interleaved=1), 2), (dict(pairs=20), 2),
    (dict(q=H(0)), 1), (dict(q=H(264)), 1), (dict(q=H(256, 12)), 1), (dict(k_out=H(256, 512, 4)), 1),
    (dict(q_weight=8), 1), (dict(positions=None), 1), (dict(inv_freq=None), 1), (dict(axes=0), 1), (dict(positions=258), 1),
    (dict(tokens=0, q=H(0)), 0), (dict(q_heads=0, k_heads=0, q=H(0), k=H(0)), 0),
])
def test_qk_norm_rope_argument_errors(lib, kw, status):
    assert lib.svdq_qk_norm_rope(ctypes.addressof(_rope(**kw)), None) == status
    assert lib.svdq_qk_norm_rope(None, None) == 1
    if status:
        assert S.svdq_last_error()


def _cache(**kw):
    base = dict(k_codes=256, k_scales=256, v_codes=256, v_scales=256, pages=8, heads=2, page_size=16, head_dim=128)
    base.update(kw)
    return S.svdq_kv4_cache(**base)


BAD_CACHES = [
    (dict(head_dim=96), 2), (dict(head_dim=256), 2), (dict(page_size=8), 2), (dict(page_size=48), 2),
    (dict(page_size=512), 2), (dict(page_size=0), 2), (dict(heads=0), 2), (dict(pages=0), 2), (dict(pages=-1), 2),
    (dict(k_codes=None), 1), (dict(v_scales=8), 1),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(lib, kw, status):
    c, h = _cache(**kw), H()
    a = ctypes.addressof
    assert lib.svdq_kv4_append(a(c), a(h), a(h), 1, 0, 256, None) == status
    assert lib.svdq_kv4_read(a(c), a(h), a(h), 1, 0, 256, None) == status
    d = _attn(cache=c)
    assert lib.svdq_kv4_attention(a(d), None, 0, None) == status
    assert lib.svdq_kv4_attention_workspace_bytes(a(d)) == 0


def test_append_and_read_argument_errors(lib):
    a, c, h, bad = ctypes.addressof, _cache(), H(), H(264)
    for fn in (lib.svdq_kv4_append, lib.svdq_kv4_read):
        assert fn(None, a(h), a(h), 1, 0, 256, None) == 1
        assert fn(a(c), None, a(h), 1, 0, 256, None) == 1
        assert fn(a(c), a(h), a(bad), 1, 0, 256, None) == 1
        assert fn(a(c), a(h), a(h), -1, 0, 256, None) == 1
        assert fn(a(c), a(h), a(h), 1, 2, 256, None) == 1
        assert fn(a(c), a(h), a(h), 1, 0, None, None) == 1
        assert fn(a(c), a(h), a(h), 1, 0, 260, None) == 1
        assert fn(a(c), a(h), a(h), 0, 0, None, None) == 0


def _attn(**kw):
    base = dict(cache=_cache(), tokens=4, requests=2, q_heads=4, dtype=0, q=H(), out=H(), kv_len=256, block_table=256,
                table_stride=4, max_pages=4, causal=1, softmax_scale=0.1)
    base.update(kw)
    return S.svdq_kv4_attention_desc(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), 1), (dict(requests=-1), 1), (dict(dtype=3), 1), (dict(softmax_scale=float("nan")), 1),
    (dict(softmax_scale=float("inf")), 1), (dict(q_heads=3), 2), (dict(q_heads=0), 2), (dict(max_pages=-1), 2),
    (dict(max_pages=1 << 28), 2), (dict(max_kv_len=-1), 2), (dict(tokens=5), 2), (dict(q=H(0)), 1),
    (dict(out=H(256, 4)), 1), (dict(kv_len=None), 1), (dict(kv_len=257), 1), (dict(block_table=None), 1),
    (dict(q_start=258), 1), (dict(lse=257), 1), (dict(tokens=0, q=H(0)), 0), (dict(requests=0, kv_len=None), 0),
])
def test_attention_argument_errors(lib, kw, status):
    assert lib.svdq_kv4_attention(ctypes.addressof(_attn(**kw)), 256, 1 << 40, None) == status
    assert lib.svdq_kv4_attention(None, None, 0, None) == 1
    assert lib.svdq_kv4_attention_workspace_bytes(None) == 0
    assert lib.svdq_kv4_attention_status(None) == 1


def test_attention_workspace_is_checked(lib):
    # One request with a long table: the key axis is split, so a workspace is needed.
    d = _attn(tokens=1, requests=1, max_pages=4096)
    need = lib.svdq_kv4_attention_workspace_bytes(ctypes.addressof(d))
    assert need > 0
    for ptr, size in ((None, need), (256, need - 1), (264, need)):
        assert lib.svdq_kv4_attention(ctypes.addressof(d), ptr, size, None) == 5


# ------------------------------------------------------------------ Python wrappers

def test_wrappers_refuse_cpu_tensors():
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    cache = S.kv4_cache(2, 16, 2, 128, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        S.qk_norm_rope(q)
    with pytest.raises(ValueError, match="CUDA"):
        S.kv4_append(cache, q, q, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        S.kv4_read(cache, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        S.kv4_attention(q, cache, torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(TypeError):
        S.qk_norm_rope([1.0])


def test_missing_extension_module_fails_loudly(lib, monkeypatch, tmp_path):
    from bit_quantized_linear_svdq_b200 import attention as A
    monkeypatch.setattr(A, "_native", None)
    monkeypatch.setattr(S, "library_path", lambda: str(tmp_path / "libsvdq_b200.so"))
    with pytest.raises(RuntimeError, match="not built"):
        A._calls()


@pytest.mark.parametrize("args", [(0, 16, 2, 128), (2, 24, 2, 128), (2, 16, 0, 128), (2, 16, 2, 96)])
def test_cache_sizes_are_checked(args):
    with pytest.raises(ValueError):
        S.kv4_cache(*args, device="cpu")


def test_rope_frequencies():
    f, axis = S.rope_frequencies((2, 3), theta=100.0, device="cpu")
    assert axis.tolist() == [0, 0, 1, 1, 1]
    torch.testing.assert_close(f.double(), torch.tensor([1, 100 ** -0.5, 1, 100 ** (-1 / 3), 100 ** (-2 / 3)],
                                                        dtype=torch.float64), rtol=2 ** -24, atol=0)
    f, axis = S.rope_frequencies((2, 2), theta=16.0, restart=False, device="cpu")
    assert f.tolist() == [1.0, 0.5, 0.25, 0.125] and axis.tolist() == [0, 0, 1, 1]
    for bad in ((), (-1,), (1.5,)):
        with pytest.raises(ValueError):
            S.rope_frequencies(bad, device="cpu")


# ------------------------------------------------------------------ which kernel takes a request

def test_every_size_of_a_call_belongs_to_one_kernel(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "kv4_plan_check")
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", B.CSRC, os.path.join(ROOT, "tests", "native", "kv4_plan_check.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert r.stdout.strip() == "ok"


@pytest.mark.parametrize("requests", [1, 2, 3, 40])
@pytest.mark.parametrize("ragged", [False, True])
def test_every_size_of_a_call_is_planned(lib, requests, ragged):
    """Over a long table each launch shares its segments among CTAs, so a call that launches anything needs a workspace."""
    for tokens in range(requests, 1100, 1 if requests == 1 else requests):
        d = _attn(tokens=tokens, requests=requests, max_pages=4096, q_start=256 if ragged else None)
        assert lib.svdq_kv4_attention_workspace_bytes(ctypes.addressof(d)) > 0, tokens


# ------------------------------------------------------------------ outputs that lie over inputs

def test_overlap_of_strided_heads(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "head_overlap_check")
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", B.CSRC, os.path.join(ROOT, "tests", "native", "head_overlap_check.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert r.stdout.strip() == "ok"


def test_more_tokens_than_the_grid_counts_are_refused(lib):
    """The grid is ceil(tokens / tokens a CTA) in 32 bits, at most 4096 tokens a CTA."""
    for tokens in (2 ** 31 - 1, 2 ** 31 - 4096):
        assert lib.svdq_qk_norm_rope(ctypes.addressof(_rope(tokens=tokens, q_heads=1, k_heads=0, head_dim=8, pairs=0)), None) == 2
