"""Index arithmetic of the 4-bit cache's attention, on the host (no GPU)."""
import os
import subprocess

import pytest
import torch

from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300 import build
from test_memory_cache import P, cache, changed, lib, refused  # noqa: F401

DIVIDE = r"""
#include <cstdio>
#include <initializer_list>
#include "cache.h"

int main() {
    const int64_t top = (int64_t(1) << 31) - 1;
    long bad = 0, n = 0;
    auto check = [&](const clef::RowDivider& d, int share, int64_t r) {
        if (r < 0 || r > top) return;
        ++n;
        bad += d(int(r)) != int(r / share);
    };
    for (int64_t base : {int64_t(1), int64_t(1) << 10, int64_t(1) << 20, int64_t(1) << 24, int64_t(1) << 30, top - 300})
        for (int64_t share = base; share < base + 300 && share <= top; ++share) {
            const clef::RowDivider d = clef::row_divider(int(share));
            for (int64_t r = 0; r < 40; ++r) {
                check(d, int(share), r);
                check(d, int(share), top - r);
                check(d, int(share), (int64_t(1) << 24) + r - 20);
                check(d, int(share), (share << 24) + r - 20);
            }
            for (int64_t q = 1; q <= top / share; q = q * 3 / 2 + 1)  // both sides of a multiple
                for (int64_t e = -1; e <= 1; ++e) check(d, int(share), q * share + e);
        }
    std::printf("%ld of %ld\n", bad, n);
    return bad != 0;
}
"""


def test_rows_are_divided_exactly(tmp_path):
    """r / share for every r that the call admits: both sides of multiples, of 2^24 and of 2^31."""
    src, exe = tmp_path / "divide.cpp", tmp_path / "divide"
    src.write_text(DIVIDE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build._nvcc())) or "/usr/local/cuda", "include")
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{build.CSRC}", f"-I{cuda}", str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout


def test_more_rows_than_32_bits_hold_are_refused():
    c = cache()
    good = [c, 2, 1 << 24, 1 << 24, 127, 0, 1, B.BF16, P, 127 * 64, 64, P, P, 4, P, 0.125, 1, P, P, P, 0, 0]
    refused(1, B.clef_cache_attend, *changed(good, 18, P + 2))              # the size is fine
    refused(3, B.clef_cache_attend, *changed(good, 4, 128))                 # 2^31 rows
    refused(3, B.clef_cache_attend, *changed(changed(changed(good, 4, 1), 2, (1 << 31) - 65535), 3, (1 << 31) - 65535))


ONCE = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"

static clef::PerDevice<int> state;
static std::atomic<int> made[200], broken;

static int get(int device, int error = 0) {
    int value = -1;
    const int e = state.get(device, &value, [&](int* v) {
        ++made[device];
        *v = device * 10;
        return error;
    });
    broken += e != error || (e == 0 && value != device * 10);
    return e;
}

int main() {
    get(3, 7);                                   // a failure is passed on ...
    get(3);                                      // ... and not kept
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([] {
            for (int i = 0; i < 20000; ++i) get(i % 5);
        });
    for (auto& t : threads) t.join();
    for (int device = 0; device < 5; ++device) broken += made[device] != (device == 3 ? 2 : 1);
    get(150);                                    // more devices than are kept
    get(150);
    broken += made[150] != 2;
    std::printf("%d\n", broken.load());
    return broken != 0;
}
"""


def test_every_device_is_prepared_once(tmp_path):
    """What attention sets up at its first call is set up for each device, and a failure is not kept."""
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(ONCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout


def test_attention_keeps_nothing_for_one_device_alone():
    """No kernel of the cache is set up once a process (a second device would be left out)."""
    for name in sorted(os.listdir(build.CSRC)):
        if name.startswith("cache"):
            with open(os.path.join(build.CSRC, name)) as f:
                assert "call_once" not in f.read(), name


def test_outputs_that_overlap_the_queries_are_refused():
    """The C entry point goes by the bytes of q, out and lse, whatever their starts and strides."""
    c = cache()
    rows, heads, row, head = 6, 8, 8 * 64 + 32, 64
    q_bytes = 2 * ((rows - 1) * row + (heads - 1) * head + 64)
    out_bytes, lse_bytes = 2 * rows * heads * 64, 4 * rows * heads
    far = P + (1 << 16)
    good = [c, 2, rows, 4, heads, 0, 4, B.BF16, P, row, head, P, P, 4, P, 0.125, 1, far, far << 1, P, 0, 0]
    for at in (P, P + 4, P + q_bytes - 4, P - out_bytes + 4):
        refused(1, B.clef_cache_attend, *changed(good, 17, at))
    for at in (P, P + q_bytes - 4, P - lse_bytes + 4, far, far + out_bytes - 4, far - lse_bytes + 4):
        refused(1, B.clef_cache_attend, *changed(good, 18, at))
    heads_first = changed(changed(good, 9, 64), 10, rows * 64)               # the same bytes, other strides
    refused(1, B.clef_cache_attend, *changed(heads_first, 17, P + 2 * rows * heads * 64 - 4))


def test_torch_outputs_that_overlap_the_queries_are_refused():
    from structured_decision_model_gb300.memory import MemoryCache
    c = MemoryCache(4, page=16, heads=2, head_dim=64, requests=3, max_len=40, device="cpu")
    cu = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(3000, dtype=torch.bfloat16)
    plain, size = (lambda at: x[at:at + 640].view(5, 2, 64)), 640
    wide = x[:5 * 200].view(5, 200)[:, :128].view(5, 2, 64)                  # rows 200 apart
    turned = x[:640].view(2, 5, 64).transpose(0, 1)                          # heads first
    for q, out in ((plain(0), plain(0)), (plain(64), plain(0)), (plain(0), plain(size - 2)), (wide, plain(100)),
                   (wide, plain(800 + 126)), (turned, plain(600)), (plain(2), turned.contiguous().set_(x, 0, (5, 2, 64)))):
        with pytest.raises(B.ClefError, match="apart from q"):
            c.attend(q, cu, 1, out=out)
    for q, out in ((plain(0), plain(size)), (wide, plain(1000)), (turned, plain(640))):
        with pytest.raises(B.ClefError, match="not on a GPU"):               # accepted so far
            c.attend(q, cu, 1, out=out)
