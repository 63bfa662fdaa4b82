"""Rules of the kernels that may be resident before the kernel ahead of them
has ended, read from their sources (no run can show that one is broken)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(__file__), "..", "mixture_experts_ffn_histogram_gb300", "csrc")


def _kernels():
    """(file, signature, body) of every kernel in the sources."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            start = text.index("{", m.start())
            depth, end = 0, start
            while True:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
                if depth == 0:
                    break
            yield os.path.basename(path), text[m.start():start], text[start:end]


def test_the_scan_sees_the_kernels():
    names = " ".join(sig for _, sig, _ in _kernels())
    for name in ("join_partials_kernel", "norm_bwd_kernel", "dense_split_kernel", "dense_pair_kernel"):
        assert name in names


def test_data_of_the_kernel_before_is_read_coherently():
    """The read-only path (a const __restrict__ pointer, __ldg) asks that data
    stay unchanged while the kernel is resident; a kernel that waits for the
    one before it is resident while that one writes.  The layer's bias, an
    input of the call, is all that may be read so."""
    waiting = [(f, sig, body) for f, sig, body in _kernels() if "wait_for_previous()" in body]
    assert len(waiting) >= 3      # the join of partial sums and the two product kernels
    for f, sig, body in waiting:
        assert "__restrict__" not in sig, f"{f}: {sig.strip()[:120]}"
        for arg in re.findall(r"__ldg\(\s*([\w.]+)", body):
            assert arg == "p.bias", f"{f}: __ldg({arg})"
