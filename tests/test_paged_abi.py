"""The paged cache's C ABI without a GPU: exports, struct layouts, sizes, and
the refusal of every argument that the host can check (none of these calls
reaches a launch)."""
import ctypes
import itertools
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "paged_kv.h")
FAKE = 0x7F0000000000   # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def sz():
    import fp8_kv_cache_amd
    return fp8_kv_cache_amd


def cache(sz, **kw):
    dtype = kw.get("dtype", 1)
    args = dict(d_k=FAKE, d_v=FAKE, page_stride=16 * 8 * 128, token_stride=8 * 128, head_stride=128, num_pages=10,
                page_size=16, kv_heads=8, head_dim=128, dtype=dtype, reserved=0)
    return sz.KvCache(**dict(args, **kw))


def batch(sz, **kw):
    args = dict(d_pages=FAKE, d_cu_tokens=FAKE, d_kv_lens=FAKE, pages_stride=5, pages_per_seq=5, num_seqs=3,
                total_tokens=6, max_tokens=4, max_kv_len=80, reserved=0)
    return sz.KvBatch(**dict(args, **kw))


def append_args(sz, **kw):
    args = dict(d_k=FAKE, d_v=FAKE, d_q=FAKE, d_q_out=FAKE, k_stride=1024, v_stride=1024, q_stride=4096,
                q_out_stride=4096, d_cos_sin=FAKE, d_q_norm=FAKE, d_k_norm=FAKE, eps=1e-6, q_heads=32, rotary_dim=128,
                max_positions=80, interleaved=0, reserved=0)
    return sz.KvAppendArgs(**dict(args, **kw))


def attention_args(sz, **kw):
    args = dict(d_q=FAKE, d_out=FAKE, d_lse=FAKE, q_stride=4096, out_stride=4096, scale=0.1, q_heads=32, causal=1,
                window=0)
    return sz.KvAttentionArgs(**dict(args, **kw))


BAD_CACHE = [dict(d_k=None), dict(d_v=None), dict(d_k=FAKE + 8), dict(d_v=FAKE + 2), dict(page_stride=16 * 8 * 128 + 4),
             dict(token_stride=1028), dict(head_stride=132), dict(token_stride=64), dict(head_stride=120),
             dict(page_stride=0), dict(token_stride=0), dict(head_stride=0), dict(page_stride=1 << 40),
             dict(num_pages=0), dict(num_pages=1 << 31), dict(page_size=0), dict(page_size=24), dict(page_size=1 << 17),
             dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=0), dict(head_dim=72), dict(head_dim=512),
             dict(dtype=0), dict(dtype=3), dict(dtype=-5), dict(reserved=1),
             dict(dtype=2, token_stride=1032)]     # E5M2: 16 bytes are 16 elements
BAD_BATCH = [dict(d_pages=None), dict(d_cu_tokens=None), dict(d_kv_lens=None), dict(d_pages=FAKE + 2),
             dict(d_cu_tokens=FAKE + 1), dict(d_kv_lens=FAKE + 3), dict(pages_stride=4), dict(pages_per_seq=0),
             dict(num_seqs=1 << 20), dict(total_tokens=1 << 24), dict(max_tokens=0), dict(max_kv_len=(1 << 31) - 1),
             dict(pages_stride=1 << 40), dict(reserved=7)]


def test_exports_are_what_the_header_declares(sz):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(kv_[a-z_0-9]+)\s*\(", text))
    assert names == {"kv_append", "kv_attention", "kv_attention_workspace_bytes", "kv_gather", "kv_scatter",
                     "kv_abi_version"}
    out = subprocess.run(["nm", "-D", "--defined-only", sz.library_path()], capture_output=True, text=True, check=True)
    exported = {line.split()[-1] for line in out.stdout.splitlines() if " T " in line}
    assert {n for n in exported if n.startswith("kv_")} == names
    assert int(re.search(r"#define KV_ABI_VERSION (\d+)u", text).group(1)) == sz.KV_ABI_VERSION


def test_struct_layouts(sz, tmp_path):
    """The binding's structs have the C structs' sizes and offsets (gcc, C99)."""
    structs = {"kv_cache": sz.KvCache, "kv_batch": sz.KvBatch, "kv_append_args": sz.KvAppendArgs,
               "kv_attention_args": sz.KvAttentionArgs}
    lines = []
    for name, s in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in s._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "paged_kv.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                        "-I", "/opt/rocm/include", str(src), "-o", str(exe)], capture_output=True, text=True)
    if r.returncode and "hip_runtime_api.h" in r.stderr:
        pytest.skip("HIP headers not usable from plain C here: " + r.stderr[:200])
    assert r.returncode == 0, r.stderr
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        what, n = line.split()
        name, _, field = what.partition(".")
        assert int(n) == (getattr(structs[name], field).offset if field else ctypes.sizeof(structs[name])), line


def calls(sz, c, b):
    yield "append", sz.kv_append(c, b, append_args(sz), stream=0)
    yield "attention", sz.kv_attention(c, b, attention_args(sz), FAKE, 1 << 40, stream=0)
    yield "gather", sz.kv_gather(c, b, FAKE, 1024, FAKE, 1024, stream=0)
    yield "scatter", sz.kv_scatter(c, b, FAKE, 1024, FAKE, 1024, stream=0)


@pytest.mark.parametrize("bad", BAD_CACHE, ids=str)
def test_every_call_refuses_a_bad_cache(sz, bad):
    for name, status in calls(sz, cache(sz, **bad), batch(sz)):
        assert status == sz.SZ_ERR_INVALID_ARGUMENT, (name, bad)
    assert sz.kv_attention_workspace_bytes(cache(sz, **bad), batch(sz), attention_args(sz)) == 0


@pytest.mark.parametrize("bad", BAD_BATCH, ids=str)
def test_every_call_refuses_a_bad_batch(sz, bad):
    for name, status in calls(sz, cache(sz), batch(sz, **bad)):
        assert status == sz.SZ_ERR_INVALID_ARGUMENT, (name, bad)
    assert sz.kv_attention_workspace_bytes(cache(sz), batch(sz, **bad), attention_args(sz)) == 0


@pytest.mark.parametrize("bad", [
    dict(d_k=None), dict(d_v=None), dict(d_k=FAKE + 2), dict(d_v=FAKE + 8), dict(d_q=FAKE + 4), dict(d_q_out=None),
    dict(d_q_out=FAKE + 8), dict(k_stride=1016), dict(v_stride=1023), dict(q_stride=4088), dict(q_out_stride=4097),
    dict(q_out_stride=8192), dict(d_cos_sin=FAKE + 4), dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=144),
    dict(rotary_dim=24), dict(max_positions=0), dict(interleaved=2), dict(d_q_norm=FAKE + 2), dict(d_k_norm=FAKE + 8),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(q_heads=0), dict(q_heads=65537),
    dict(reserved=1)], ids=str)
def test_append_refuses(sz, bad):
    assert sz.kv_append(cache(sz), batch(sz), append_args(sz, **bad), stream=0) == sz.SZ_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bad", [
    dict(d_q=None), dict(d_out=None), dict(d_q=FAKE + 8), dict(d_out=FAKE + 2), dict(d_lse=FAKE + 2),
    dict(q_stride=4088), dict(out_stride=4100), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
    dict(scale=float("nan")), dict(q_heads=0), dict(q_heads=12), dict(q_heads=8 * 65, q_stride=1 << 20, out_stride=1 << 20),
    dict(causal=2), dict(causal=0, window=5), dict(window=1 << 31)], ids=str)
def test_attention_refuses(sz, bad):
    a = attention_args(sz, **bad)
    assert sz.kv_attention(cache(sz), batch(sz), a, FAKE, 1 << 40, stream=0) == sz.SZ_ERR_INVALID_ARGUMENT
    assert sz.kv_attention_workspace_bytes(cache(sz), batch(sz), a) == 0


def test_other_refusals(sz):
    E = sz.SZ_ERR_INVALID_ARGUMENT
    c, b = cache(sz), batch(sz)
    for status in (FAKE + 1, FAKE + 2):
        assert sz.kv_append(c, b, append_args(sz), status, stream=0) == E
        assert sz.kv_attention(c, b, attention_args(sz), FAKE, 1 << 40, status, stream=0) == E
        assert sz.kv_gather(c, b, FAKE, 1024, FAKE, 1024, status, stream=0) == E
    for call in (sz.kv_gather, sz.kv_scatter):
        for args in itertools.product((None, FAKE, FAKE + 8), (1024, 1016, 1028), (None, FAKE), (1024, 0)):
            if args not in ((FAKE, 1024, FAKE, 1024),):
                assert call(c, b, *args, stream=0) == E, args
    assert sz._lib.kv_append(None, ctypes.addressof(b), ctypes.addressof(append_args(sz)), None, None) == E
    assert sz._lib.kv_append(ctypes.addressof(c), None, ctypes.addressof(append_args(sz)), None, None) == E
    assert sz._lib.kv_append(ctypes.addressof(c), ctypes.addressof(b), None, None, None) == E
    assert sz._lib.kv_attention(ctypes.addressof(c), ctypes.addressof(b), None, FAKE, 1, None, None) == E


def test_attention_workspace(sz):
    """Long lengths need a workspace (missing: refused; short: too small),
    one short sequence none; sizes are a function of the shapes."""
    long = batch(sz, num_seqs=1, total_tokens=1, max_tokens=1, max_kv_len=100000, pages_per_seq=7000, pages_stride=7000)
    a = attention_args(sz)
    need = sz.kv_attention_workspace_bytes(cache(sz), long, a)
    assert need >= 2 * 32 * (128 + 2) * 4 and need % 256 == 0
    assert sz.kv_attention(cache(sz), long, a, None, need, stream=0) == sz.SZ_ERR_INVALID_ARGUMENT
    assert sz.kv_attention(cache(sz), long, a, FAKE + 8, need, stream=0) == sz.SZ_ERR_INVALID_ARGUMENT
    assert sz.kv_attention(cache(sz), long, a, FAKE, need - 1, stream=0) == sz.SZ_ERR_BUFFER_TOO_SMALL
    short = batch(sz, num_seqs=1, total_tokens=1, max_tokens=1, max_kv_len=33)
    assert sz.kv_attention_workspace_bytes(cache(sz), short, a) == 0


def test_nothing_to_do_is_no_error(sz):
    """No sequences or no rows: OK, and no table or tensor is looked at."""
    for b in (batch(sz, num_seqs=0, d_pages=None, d_cu_tokens=None, d_kv_lens=None),
              batch(sz, total_tokens=0, max_tokens=0, d_pages=None)):
        assert sz.kv_append(cache(sz), b, append_args(sz, d_k=None, d_q=None, d_q_norm=None), stream=0) == sz.SZ_OK
        assert sz.kv_attention(cache(sz), b, attention_args(sz, d_q=None, d_out=None), None, 0, stream=0) == sz.SZ_OK
        assert sz.kv_gather(cache(sz), b, None, 0, None, 0, stream=0) == sz.SZ_OK
        assert sz.kv_scatter(cache(sz), b, None, 0, None, 0, stream=0) == sz.SZ_OK


def test_the_tensor_layer_refuses_on_the_host(sz):
    """Host tensors, and tensors of other shapes, never reach the library."""
    import torch
    from fp8_kv_cache_amd import paged
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(sz.SzError):
        paged.PagedCache(k, k)
    with pytest.raises(sz.SzError):
        paged.PagedCache(k, k[:, :8])
    with pytest.raises(sz.SzError):
        paged.PagedCache(k.float(), k.float())
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(sz.SzError):
        paged.PageBatch(one[None], torch.zeros(2, dtype=torch.int32), one)
    with pytest.raises(sz.SzError):
        paged.Rope(torch.zeros(4, 16))


def test_library_is_one_and_device_code_has_no_packed_fp32(sz):
    """The kernels compiled to gfx950 assembly with the build's flags: the
    attention is on the matrix cores, nothing spills its loop to scratch
    in the common dimensions, and no packed FP32 instruction is there."""
    import importlib.util
    spec = importlib.util.spec_from_file_location("_paged_build", os.path.join(ROOT, "fp8_kv_cache_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for name in ("kv_kernels.hip", "kv_attention.hip"):
        cmd = [mod.hipcc(), *mod.flags(), "--cuda-device-only", "-S", "-o", "-", os.path.join(ROOT, "fp8_kv_cache_amd", "csrc", name)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        instructions = [ln.split()[0] for ln in r.stdout.splitlines() if re.match(r"\s+[sv]_\w+", ln)]
        assert not [i for i in instructions if i in ("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32")]
        assert any(i.startswith("v_mfma") for i in instructions) == (name == "kv_attention.hip")


def test_attention_in_place_wants_one_stride(sz):
    """A row written into the query's place must not be another row's query."""
    for strides in (dict(q_stride=8192), dict(out_stride=8192)):
        a = attention_args(sz, **strides)
        assert sz.kv_attention(cache(sz), batch(sz), a, FAKE, 1 << 40, stream=0) == sz.SZ_ERR_INVALID_ARGUMENT
        assert sz.kv_attention_workspace_bytes(cache(sz), batch(sz), a) == 0
    apart = attention_args(sz, d_out=FAKE + (1 << 20), out_stride=8192)
    long = batch(sz, num_seqs=1, total_tokens=1, max_tokens=1, max_kv_len=100000, pages_per_seq=7000, pages_stride=7000)
    assert sz.kv_attention_workspace_bytes(cache(sz), long, apart) > 0
    # one token has one row, whatever its stride
    assert sz.kv_attention_workspace_bytes(cache(sz), long, attention_args(sz, out_stride=8192)) > 0
