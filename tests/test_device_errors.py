"""Device error words of all translation units: each is read (and so cleared)
by every query, and the first that is set is reported.  The readers are fakes."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_int8_linear_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "device_errors.h"

unsigned words[4];
bool fails[4];
template <int I>
int read(unsigned* code) {
    if (fails[I]) return 1;
    *code = words[I];
    words[I] = 0;
    return 0;
}

int main() {
    int (*const readers[])(unsigned*) = {read<0>, read<1>, read<2>, read<3>};
    unsigned code = 77;
    auto query = [&] { return w8a8::read_device_errors(readers, &code); };
    if (query() != 0 || code != 0) return 1;                   // nothing set
    words[1] = 0x132, words[2] = 0x145, words[3] = 1;
    if (query() != 0 || code != 0x132) return 2;               // the first
    for (unsigned w : words)
        if (w) return 3;                                       // all were read
    if (query() != 0 || code != 0) return 4;                   // and nothing is left
    words[0] = 0x140, words[3] = 0x150, fails[1] = true;
    if (query() == 0) return 5;                                // a read that fails is reported,
    if (words[3] != 0) return 6;                               // and the others are still cleared
    return 0;
}
"""


def test_every_word_is_read(tmp_path):
    (tmp_path / "t.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "t")
    subprocess.run(["g++", "-std=c++17", "-I" + CSRC, str(tmp_path / "t.cpp"), "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0


def test_the_library_reads_them_so():
    with open(os.path.join(CSRC, "api.cu")) as f:
        api = f.read()
    body = api[api.index("w8a8_status w8a8_get_device_error"):]
    body = body[:body.index("\n}")]
    assert "read_device_errors(" in body
    for unit in ("gemm", "gemm_s8", "quant", "attention", "attention_split", "residual_norm"):
        assert f"w8a8::{unit}_read_device_error" in body, unit
