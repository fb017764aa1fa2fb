"""CPU checks of the paged-cache calls: struct layouts, every refusal that the
header documents (returned before anything is launched), and the index
arithmetic that the kernels share with the host: division by the page size,
clamped rows and lengths, and slots of page tables with bad ids."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

import kv_cache_compression_decode_amd as kvc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a well-aligned address; a refused call never touches it
INVALID, SHAPE, CAPACITY = kvc.ERR_INVALID_ARG, kvc.ERR_SHAPE, kvc.ERR_CAPACITY


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kvc.LIB_PATH):
        from kv_cache_compression_decode_amd import build

        build.build()
    return kvc.lib()


def _desc(**kw):
    f = dict(n_layers=2, n_heads=8, n_kv_heads=2, head_dim=128, page_tokens=16, n_pages=100,
             cache_dtype=0, io_dtype=0)
    f.update(kw)
    return kvc.PagedDesc(*f.values())


def _batch(**kw):
    f = dict(table=A, lens=A, q_start=None, n_seqs=3, table_stride=10, n_tokens=3, max_len=160)
    f.update(kw)
    return kvc._PagedBatch(*f.values())


def test_struct_layouts():
    assert ctypes.sizeof(kvc.PagedDesc) == 32
    assert ctypes.sizeof(kvc._PagedBatch) == 40
    assert kvc._PagedBatch.n_seqs.offset == 24
    assert ctypes.sizeof(kvc._RopeArgs) == 24


@pytest.mark.parametrize("bad", [
    dict(n_layers=0), dict(n_layers=32768), dict(n_heads=0), dict(n_kv_heads=0),
    dict(n_heads=9), dict(n_heads=258, n_kv_heads=2), dict(n_heads=4224, n_kv_heads=64),
    dict(head_dim=0), dict(head_dim=80), dict(head_dim=512), dict(page_tokens=0), dict(n_pages=0),
    dict(page_tokens=1 << 16, n_pages=1 << 15), dict(cache_dtype=2), dict(io_dtype=2),
    dict(cache_dtype=1, io_dtype=0)])
def test_descriptor_refusals(L, bad):
    assert L.kvc_validate_paged_desc(_desc(**bad)) == INVALID
    assert L.kvc_attend_ws_bytes(_desc(**bad), _batch()) == 0
    assert _append(L, _desc(**bad)) == INVALID
    assert _attend(L, _desc(**bad)) == INVALID
    assert _page(L, _desc(**bad)) == INVALID


def test_descriptor_accepted(L):
    for d in (64, 96, 128, 256):
        for c, i in ((0, 0), (1, 1), (0, 1)):
            assert L.kvc_validate_paged_desc(_desc(head_dim=d, cache_dtype=c, io_dtype=i)) == 0
    assert L.kvc_validate_paged_desc(_desc(n_heads=128, n_kv_heads=1, page_tokens=1500)) == 0
    assert L.kvc_validate_paged_desc(None) == INVALID


def _append(L, d=None, b=None, layer=0, pool=A, k=A, ks=256, v=A, vs=256, q=A, qs=1024, o=A,
            os_=1024, rope=None, status=A):
    return L.kvc_append(d or _desc(), b or _batch(), layer, pool, k, ks, v, vs, q, qs, o, os_,
                        rope, status, None)


def _attend(L, d=None, b=None, layer=0, pool=A, q=A, qs=1024, scale=1.0, window=0, o=A, os_=1024,
            lse=A, ws=A, ws_bytes=1 << 40, status=A, name="kvc_attend"):
    return getattr(L, name)(d or _desc(), b or _batch(), layer, pool, q, qs, scale, window, o, os_,
                            lse, ws, ws_bytes, status, None)


def _page(L, d=None, pool=A, table=A, entries=10, first=0, n=100, flat=1 << 40, T=200, at=0,
          status=A, name="kvc_page_out"):
    d = d or _desc()
    if name == "kvc_page_out":
        return L.kvc_page_out(d, pool, table, entries, first, n, flat, T, at, status, None)
    return L.kvc_page_in(d, flat, T, at, pool, table, entries, first, n, status, None)


BATCH_BAD = [
    (dict(n_seqs=(1 << 20) + 1, n_tokens=(1 << 20) + 1), SHAPE),
    (dict(n_tokens=4), SHAPE),
    (dict(max_len=161), SHAPE),
    (dict(table_stride=1 << 27, max_len=(1 << 30) + 1), SHAPE),
    (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(lens=A + 2), INVALID),
    (dict(table=A + 1), INVALID), (dict(q_start=A + 2), INVALID),
    (dict(q_start=A, n_tokens=(1 << 20) + 1), SHAPE)]


@pytest.mark.parametrize("bad,code", BATCH_BAD)
def test_batch_refusals(L, bad, code):
    b = _batch(**bad)
    assert _append(L, b=b) == code
    assert _attend(L, b=b, name="kvc_attend_prompt" if b.q_start else "kvc_attend") == code


def test_append_refusals(L):
    assert _append(L, layer=2) == SHAPE
    for p in ("pool", "k", "v", "status"):
        assert _append(L, **{p: None}) == INVALID
        assert _append(L, **{p: A + 2}) == INVALID
    for p in ("q", "o"):
        assert _append(L, **{p: None}) == INVALID  # q and q_out go together
        assert _append(L, **{p: A + 8}) == INVALID
    for s, least in (("ks", 256), ("vs", 256), ("qs", 1024), ("os_", 1024)):
        assert _append(L, **{s: least + 4}) == INVALID
        assert _append(L, **{s: least - 8}) == SHAPE
    assert _append(L, qs=2048) == SHAPE  # in place with two strides

    def rope(cos_sin=A, n=200, dim=128, inter=0, reserved=0):
        return kvc._RopeArgs(cos_sin, n, dim, inter, reserved)
    for r in (rope(None), rope(A + 4), rope(dim=0), rope(dim=8), rope(dim=24), rope(dim=144),
              rope(inter=2), rope(reserved=1)):
        assert _append(L, rope=r) == INVALID


def test_attend_refusals(L):
    assert _attend(L, layer=2) == SHAPE
    for p in ("pool", "q", "o", "status"):
        assert _attend(L, **{p: None}) == INVALID
        assert _attend(L, **{p: A + 2}) == INVALID
    assert _attend(L, lse=A + 2) == INVALID
    assert _attend(L, qs=1020) == INVALID and _attend(L, os_=1016) == SHAPE
    for s in (float("inf"), float("nan"), float("-inf")):
        assert _attend(L, scale=s) == INVALID
    long = _batch(table_stride=10000, max_len=100000)
    need = L.kvc_attend_ws_bytes(_desc(), long)
    assert need > 0
    assert _attend(L, b=long, ws_bytes=need - 1) == CAPACITY
    assert _attend(L, b=long, ws=None) == INVALID
    assert _attend(L, b=long, ws=A + 128) == INVALID
    # each form refuses the other's batch
    assert _attend(L, b=_batch(q_start=A)) == INVALID
    assert _attend(L, name="kvc_attend_prompt") == INVALID
    big = _batch(q_start=A, n_tokens=1 << 20)
    assert _attend(L, d=_desc(n_heads=16), b=big, qs=2048, os_=2048,
                   name="kvc_attend_prompt") == SHAPE


@pytest.mark.parametrize("name", ["kvc_page_out", "kvc_page_in"])
def test_page_refusals(L, name):
    assert _page(L, n=161, T=300, name=name) == SHAPE
    assert _page(L, first=61, name=name) == SHAPE
    assert _page(L, first=(1 << 32) - 1, name=name) == SHAPE
    assert _page(L, T=99, name=name) == SHAPE
    assert _page(L, at=101, name=name) == SHAPE
    assert _page(L, n=(1 << 27) + 1, entries=(1 << 24), T=1 << 28, name=name) == SHAPE
    assert _page(L, flat=A + 4096, name=name) == SHAPE  # overlaps the pool
    for p in ("pool", "table", "flat", "status"):
        assert _page(L, **{p: None}, name=name) == INVALID
        assert _page(L, **{p: A + 2}, name=name) == INVALID


def test_empty_calls_do_nothing(L):
    none = _batch(n_seqs=0, n_tokens=0, table=None, lens=None)
    assert _append(L, b=none) == 0 and _attend(L, b=none) == 0
    for q_start in (None, A):
        for n in (0, 3):
            b = _batch(n_seqs=n, n_tokens=0, q_start=q_start)
            assert L.kvc_attend_ws_bytes(_desc(), b) == 0
    assert _attend(L, b=_batch(q_start=A, n_tokens=0), name="kvc_attend_prompt") == 0
    assert _page(L, n=0) == 0 and _page(L, n=0, name="kvc_page_in") == 0


def test_binding_refusals():
    with pytest.raises(kvc.KvcError):
        kvc.make_paged_desc(1, 8, 2, 80, 16, 4)
    with pytest.raises(kvc.KvcError):
        kvc.make_paged_desc(1, 8, 2, 64, 16, 4, cache_dtype=torch.float32)
    t = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError):  # host tensors
        kvc.PagedBatch(t, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvc.Rope(torch.zeros((4, 16)))


HOST = r"""
#include <cstdio>
#include <cstdlib>
#include "kvc_paged.h"
using namespace kvc;
#define CHECK(x) \
  do { if (!(x)) { std::printf("failed: %s, line %d\n", #x, __LINE__); return 1; } } while (0)
int main() {
  // the quotient, at multiples of the divisor and next to them
  uint32_t ds[] = {1, 2, 3, 5, 7, 10, 16, 20, 48, 1000, 1500, 4097, 65535, 65536, 65537,
                   (1u << 30) - 1, 1u << 30, (1u << 30) + 1, (1u << 31) - 1, 1u << 31};
  for (uint32_t d : ds) {
    const FastDiv f = FastDiv::make(d);
    const uint32_t top = (1u << 31) - 1;
    for (uint64_t k = 0; k < 3000; ++k) {
      const uint64_t base = (k < 1500 ? k : (uint64_t)top / d - (k - 1500)) * d;
      for (int e = -2; e <= 2; ++e) {
        const uint64_t n = base + (uint64_t)(int64_t)e;
        if (n <= top) CHECK(f.div((uint32_t)n) == (uint32_t)n / d);
      }
    }
    uint32_t x = 12345;
    for (int i = 0; i < 100000; ++i) {
      x = x * 1664525u + 1013904223u;
      CHECK(f.div(x >> 1) == (x >> 1) / d);
    }
  }
  // slots: ids outside the pool give false and a slot inside it
  const int32_t table[] = {4, -1, 0, 5, 1000000, (int32_t)0x80000000, 3};
  Seqs pool{};
  pool.page = FastDiv::make(20);
  pool.n_pages = 5;
  for (uint32_t j = 0; j < 140; ++j) {
    uint32_t slot = 0xFFFFFFFFu;
    const int32_t id = table[j / 20];
    const bool ok = pool.slot_of(table, j, slot);
    CHECK(ok == (id >= 0 && id < 5));
    CHECK(slot < 100);
    if (ok) CHECK(slot == (uint32_t)id * 20 + j % 20);
  }
  // rows and lengths: clamped to the batch whatever the device arrays hold
  const int32_t big = 0x7FFFFFFF, low = (int32_t)0x80000000;
  const int32_t starts[] = {0, 5, 3, -7, 40, 9, big, low, 12, 12};
  const int32_t lens[] = {0, 7, -1, 100, 101, big, low, 50, 3};
  Seqs s{};
  s.lens = lens;
  s.q_start = starts;
  s.n_seqs = 9;
  s.n_tokens = 12;
  s.max_len = 100;
  for (uint32_t b = 0; b < 9; ++b) {
    uint32_t row, n;
    s.rows(b, row, n);
    CHECK(row <= 12 && row + n <= 12);
    const bool good = starts[b] >= 0 && starts[b] <= starts[b + 1] && starts[b + 1] <= 12;
    CHECK(s.rows_bad(b) == !good);
    if (good) CHECK((int32_t)row == starts[b] && (int32_t)n == starts[b + 1] - starts[b]);
    CHECK(s.len(b) >= 0 && s.len(b) <= 100);
    CHECK(s.len_bad(b) == (lens[b] < 0 || lens[b] > 100));
    if (!s.len_bad(b)) CHECK(s.len(b) == lens[b]);
  }
  s.q_start = nullptr;
  uint32_t row, n;
  s.rows(6, row, n);
  CHECK(row == 6 && n == 1 && !s.rows_bad(6));
  std::puts("ok");
  return 0;
}
"""


def test_index_arithmetic_on_the_host(tmp_path):
    """The kernels' own index functions, compiled for the host."""
    from kv_cache_compression_decode_amd import build

    src = tmp_path / "index.hip"
    src.write_text(HOST)
    exe = tmp_path / "index"
    subprocess.check_call([build.hipcc(), "-O1", "-std=c++17", "--offload-host-only",
                           "-I", os.path.join(ROOT, "include"), "-I", build.CSRC, str(src),
                           "-o", str(exe)])
    assert subprocess.check_output([str(exe)], text=True).strip() == "ok"


class _HostBatch:
    """Stands for a batch whose tensors are in host memory: the binding's
    checks can be walked without a GPU."""
    device = torch.device("cpu")
    n_seqs = 1

    def _args(self, desc, n):
        return _batch(n_seqs=1, n_tokens=n)


class _Scratch:
    def __init__(self, ws, status):
        self.ws, self.status = ws, status
        self.ws_bytes = ws.numel()


@pytest.mark.parametrize("call", ["append_async", "attend_async", "attend_prompt_async"])
@pytest.mark.parametrize("elsewhere", ["ws", "status"])
def test_workspace_of_another_device(call, elsewhere):
    """A workspace or status word on another device than the batch would be
    written through an address that means something else there."""
    desc = _desc(n_layers=1, n_heads=4, head_dim=64, n_pages=2)
    host = dict(ws=torch.zeros(256, dtype=torch.uint8), status=torch.zeros(1, dtype=torch.int32))
    host[elsewhere] = host[elsewhere].to("meta")
    wsp = _Scratch(**host)
    pool = torch.zeros(desc.pool_shape, dtype=torch.float16)
    q = torch.zeros((1, 4, 64), dtype=torch.float16)
    k = torch.zeros((1, 2, 64), dtype=torch.float16)
    args = (k, k) if call == "append_async" else (q, q.clone())
    with pytest.raises(ValueError, match="workspace"):
        getattr(kvc, call)(desc, _HostBatch(), 0, pool, *args, wsp)


@pytest.mark.parametrize("cache,other", [(0, torch.bfloat16), (1, torch.float16)])
def test_page_moves_check_the_tensors_type(cache, other):
    """Page moves copy bits, so a tensor of the other 16-bit type (or one that
    is not [L][2][T][C]) is refused; bit patterns go with either type."""
    desc = _desc(n_layers=1, head_dim=64, n_pages=2, cache_dtype=cache, io_dtype=cache)
    pool = torch.zeros(desc.pool_shape, dtype=kvc._DTYPES[cache])
    table = torch.zeros(2, dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32)

    def both(flat, match):
        with pytest.raises(ValueError, match=match):
            kvc.page_out_async(desc, pool, table, 0, 5, flat, 0, status)
        with pytest.raises(ValueError, match=match):
            kvc.page_in_async(desc, flat, 0, pool, table, 0, 5, status)

    good = torch.zeros((1, 2, 5, 128), dtype=pool.dtype)
    for t in (other, torch.uint16):
        both(good.to(t), "type")
    both(good[0, 0], "dimension")
    # past these checks: refused for lying in host memory
    both(good, "CUDA")
    both(good.view(torch.int16), "CUDA")


@pytest.mark.parametrize("name", ["kvc_attend", "kvc_attend_prompt"])
def test_scales_that_pass_the_range(L, name):
    """The kernels take scale * log2(e) in binary32, below 2^128: a scale of
    2^128 / log2(e) = 2.3586e38 and above would make every score an infinity or NaN."""
    q_start = A if name == "kvc_attend_prompt" else None
    some = _batch(q_start=q_start)
    none = _batch(n_seqs=0, n_tokens=0, q_start=q_start)  # accepted, nothing is launched
    for s in (2.359e38, 2.9e38, 3.4e38, float("inf"), float("nan")):
        for sign in (1.0, -1.0):
            assert _attend(L, b=some, scale=sign * s, name=name) == INVALID
            assert _attend(L, b=none, scale=sign * s, name=name) == INVALID
    for s in (2.358e38, 1.0, 1e-45, 0.0):
        for sign in (1.0, -1.0):
            assert _attend(L, b=none, scale=sign * s, name=name) == 0


@pytest.mark.parametrize("name", ["kvc_attend", "kvc_attend_prompt"])
def test_attention_in_place_with_two_strides(L, name):
    """With out at q's place, row i of out must be row i of q: at another
    stride it lies on rows whose queries are still to be read."""
    b = _batch(q_start=A if name == "kvc_attend_prompt" else None)
    big = 1 << 40
    assert _attend(L, b=b, qs=2048, os_=1024, ws_bytes=big, name=name) == SHAPE
    assert _attend(L, b=b, qs=1024, os_=1032, ws_bytes=big, name=name) == SHAPE


def test_workspace_bound(L):
    """The header's bound over every batch of a descriptor; the size itself is
    not monotone (a long prompt fills the chip uncut and needs nothing)."""
    r = random.Random(5)
    most = {}
    for _ in range(20000):
        d = r.choice([64, 96, 128, 256])
        kv = r.choice([1, 2, 3, 4, 5, 8, 16, 64, 512])
        group = r.choice([1, 2, 4, 7, 8, 16, 17, 64, 128])
        if kv * group > 4096:
            continue
        n_seqs = int(2 ** r.uniform(0, 20)) if r.random() < 0.3 else r.randint(1, 600)
        q_start = r.choice([None, A])
        n_tokens = int(2 ** r.uniform(0, 20)) if q_start else n_seqs
        b = _batch(n_seqs=n_seqs, n_tokens=n_tokens, q_start=q_start, table_stride=1 << 26,
                   max_len=int(2 ** r.uniform(0, 30)))
        need = L.kvc_attend_ws_bytes(_desc(head_dim=d, n_heads=kv * group, n_kv_heads=kv), b)
        assert need <= 65536 * (4 * d + 8) + 16640, (d, kv, group, n_seqs, n_tokens, b.max_len)
        most[d] = max(most.get(d, 0), need)
    for d in (64, 96, 128):  # the bound is met, but for the join's records
        assert most[d] >= 65536 * (4 * d + 8)
    sizes = [L.kvc_attend_ws_bytes(_desc(n_heads=64, n_kv_heads=8), _batch(
        n_seqs=1, n_tokens=n, q_start=A, table_stride=1000, max_len=16000)) for n in (37, 9000)]
    assert sizes[0] > sizes[1] == 0
