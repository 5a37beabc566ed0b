"""The lists of adjust_logits (a row's part of the history and of the biases)
where their numbers are near the ends of int: cut to the list before anything
is computed from them.  The cut is tried on the CPU, as C++ of its own; what
the kernel then does with such rows on the GPU."""
import ctypes
import itertools
import os
import subprocess

import pytest
import torch

from tests.test_adjust_logits import DEV, Case, run

LOW, HIGH = -(1 << 31), (1 << 31) - 1
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_streaming_expert_gb300", "csrc")
NUMBERS = sorted({e + d for e in (0, 7, 1000) for d in (-2, -1, 0, 1, 2)} | {LOW + d for d in range(3)} |
                 {HIGH - d for d in (0, 1, 100, 254, 255, 256, 2048)})


@pytest.fixture(scope="module")
def cuts(tmp_path_factory):
    at = tmp_path_factory.mktemp("cuts")
    (at / "cuts.cpp").write_text("""
        #include "list_parts.h"
        extern "C" void span(int begin, int answer, int end, int n, int* out) {
          const wse::Span s = wse::cut_span(begin, answer, end, n);
          out[0] = s.begin, out[1] = s.answer, out[2] = s.end;
        }
        extern "C" void part(int from, int to, int n, int* out) {
          const wse::Part p = wse::cut_part(from, to, n);
          out[0] = p.from, out[1] = p.to;
        }
        """)
    # overflowing signed arithmetic ends the compiled function
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-ftrapv", "-I", CSRC, str(at / "cuts.cpp"), "-o",
                    str(at / "cuts.so")], check=True)
    return ctypes.CDLL(str(at / "cuts.so"))


def test_spans_are_cut_to_the_history(cuts):
    out = (ctypes.c_int * 3)()
    for n in (0, 1, 7, 1000, HIGH):
        for begin, answer, end in itertools.product(NUMBERS, repeat=3):
            cuts.span(begin, answer, end, n, out)
            b, a, e = out
            assert 0 <= b <= a <= e <= n
            # what any reading of the header's words leaves: the positions in both
            want = range(max(begin, 0), min(end, n))
            assert e - b == len(want) and (not want or (b, e) == (want[0], want[-1] + 1))
            made = range(max(begin, answer, 0), min(end, n))
            assert e - a == len(made)


def test_bias_starts_are_cut_to_the_list(cuts):
    out = (ctypes.c_int * 2)()
    for n in (0, 1, 7, 1000, HIGH):
        for start, end in itertools.product(NUMBERS, repeat=2):
            cuts.part(start, end, n, out)
            assert 0 <= out[0] <= out[1] <= n
            want = range(max(start, 0), min(end, n))
            assert out[1] - out[0] == len(want) and (not want or out[0] == want[0])


@pytest.mark.gpu
def test_spans_near_the_ends_of_int():
    history = list(range(40)) * 20
    n = len(history)
    spans = [(HIGH, HIGH, 5), (HIGH, 0, 0), (0, 0, LOW), (5, 9, LOW), (HIGH, LOW, LOW), (LOW, LOW, HIGH), (LOW, HIGH, HIGH),
             (HIGH - 1, HIGH, HIGH), (0, LOW, n), (0, HIGH, n), (LOW, 100, HIGH), (n, n, HIGH), (LOW, LOW, LOW)]
    run(Case(len(spans), 50, spans, history, seed=21))


@pytest.mark.gpu
def test_bias_starts_near_the_ends_of_int():
    from weight_streaming_expert_gb300 import adjust_logits
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    starts = (HIGH, 2, HIGH - 254, HIGH, LOW, LOW, HIGH, HIGH - 1, LOW, 1)
    ids, values = list(range(300)), [float(i + 1) for i in range(300)]
    M = len(starts) - 1
    got = adjust_logits(torch.zeros(M, 310, device=DEV), bias_ids=i32(*ids), bias_values=torch.tensor(values, device=DEV),
                        bias_starts=i32(*starts)).cpu()
    want = torch.zeros(M, 310)
    for m in range(M):
        for i in range(max(starts[m], 0), min(starts[m + 1], 300)):
            want[m, ids[i]] = values[i]
    assert want[1].any() and want[5].any() and torch.equal(got, want)
