"""The check of clipped tensors for overlaps, without a GPU: what it finds, and that it says so where it gets no memory
(an exception would end the caller's process at the library's C entry)."""
import os
import shutil
import subprocess

import pytest

from text_embedding_encoder_gb300 import build

SOURCE = r"""
#include "clip_ranges.h"
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static bool refuse = false;
void* operator new(size_t n) { if (refuse) throw std::bad_alloc(); return malloc(n); }
void* operator new[](size_t n) { if (refuse) throw std::bad_alloc(); return malloc(n); }
void* operator new(size_t n, const std::nothrow_t&) noexcept { return refuse ? nullptr : malloc(n); }
void* operator new[](size_t n, const std::nothrow_t&) noexcept { return refuse ? nullptr : malloc(n); }
void operator delete(void* p) noexcept { free(p); }
void operator delete[](void* p) noexcept { free(p); }
void operator delete(void* p, size_t) noexcept { free(p); }
void operator delete[](void* p, size_t) noexcept { free(p); }

static int check(int n, const long long* rows, bool with_outs) {   // rows: {gradient, count, type, out}
    const void* grads[8];
    void* outs[8];
    int64_t counts[8];
    int32_t types[8];
    for (int i = 0; i < n; ++i) {
        grads[i] = (const void*)rows[4 * i], counts[i] = rows[4 * i + 1], types[i] = (int)rows[4 * i + 2];
        outs[i] = (void*)rows[4 * i + 3];
    }
    return clip_overlaps(grads, counts, types, 1, with_outs ? outs : nullptr, n);
}

int main() {
    const long long apart[] = {1000, 100, 0, 1000, 1400, 50, 1, 1400, 9000, 0, 0, 1000};
    const long long touching[] = {1000, 101, 0, 1000, 1400, 50, 1, 1400};
    const long long onto_other[] = {1000, 100, 0, 5000, 5396, 50, 1, 7000};
    const long long beside[] = {1000, 100, 0, 5000, 5400, 50, 1, 7000};
    const long long shared_gradient[] = {1000, 100, 0, 5000, 1000, 100, 0, 6000};
    const long long shared_output[] = {1000, 100, 0, 5000, 2000, 100, 0, 5000};
    printf("%d %d %d ", check(0, apart, false), check(3, apart, false), check(3, apart, true));
    printf("%d %d %d ", check(2, touching, false), check(2, onto_other, true), check(2, beside, true));
    printf("%d %d ", check(2, shared_gradient, true), check(2, shared_output, true));
    refuse = true;
    const int without = check(3, apart, true);
    refuse = false;
    printf("%d\n", without);
}
"""


def test_overlaps_and_no_memory(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    (tmp_path / "t.cpp").write_text(SOURCE)
    exe = os.path.join(tmp_path, "t")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", build.CSRC, str(tmp_path / "t.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["0", "0", "0", "1", "1", "0", "0", "1", "-1"]
