"""Kernels that may be set up while the stream's last kernel is still running: what that kernel may still write is not
read through the path for data that nobody writes while a kernel runs."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_draft_lm_gb300",
                    "csrc")
# inputs that are complete before the launch in front of the kernel starts
COMPLETE = {("k_sort_cluster", "tokens")}


def _kernels():
    """(file, name, signature, body) of the training and update kernels that wait for the kernel before."""
    for path in sorted(glob.glob(os.path.join(CSRC, "train_*.cu")) + glob.glob(os.path.join(CSRC, "optim_*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for part in re.split(r"\b__global__\b", text)[1:]:
            head, body = part.split("{", 1)
            if "pdl_wait()" in body:
                yield os.path.basename(path), re.search(r"(k_\w+)\(", head).group(1), head, body


def test_the_kernels_are_found():
    assert {k[1] for k in _kernels()} >= {"k_scores", "k_scores_backward", "k_scores_step", "k_adamw8", "k_adamw32",
                                          "k_norm", "k_fill", "k_sum_runs", "k_join_runs"}


def test_nothing_is_promised_that_the_kernel_before_may_write():
    for path, name, head, _ in _kernels():
        promised = set(re.findall(r"\bconst\s+\w+\s*\*\s*__restrict__\s+(\w+)", head))
        assert not {(name, p) for p in promised} - COMPLETE, (path, name, promised)


def test_no_read_only_loads():
    for path in sorted({k[0] for k in _kernels()}):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, path)).read())
        assert not re.search(r"\b__ldg\(|\bld\.global\S*\.nc\b", text), path
