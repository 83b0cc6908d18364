"""What the choice's source must keep to.  Its threads leave together or not at all: those that go
on would use what the others were to write.  And a counter in shared memory that threads read is not set
back before a barrier behind those reads (a warp that came late would read 0 and take another way
than the others, through other barriers)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bwd_sparse_mqa_gb300", "csrc")
BARRIER = r"__syncthreads\(\)|template reduce<|exact_scores<[^;]*>\(tk, some"
# (settle sets it back before its first barrier.)
RESET = r"misc\[3\] = 0|settle\(tk"
READ = r"misc\[3\](?! =)"


def _events(code):
    """Reads, resets and barriers in the order of the text, which is that of the calls here."""
    return [(m.lastgroup, m.start()) for m in re.finditer(f"(?P<barrier>{BARRIER})|(?P<reset>{RESET})|(?P<read>{READ})", code)]


def _early_resets(code):
    code = re.sub(r"//[^\n]*", "", code)
    open_read, bad = None, []
    for kind, at in _events(code):
        if kind == "barrier":
            open_read = None
        elif kind == "read":
            open_read = at
        elif open_read is not None:
            bad.append(code.count("\n", 0, at) + 1)
    return bad


def test_the_counter_is_read_before_it_is_set_back():
    with open(os.path.join(CSRC, "smqa_topk.cu")) as f:
        code = f.read()
    kinds = [k for k, _ in _events(re.sub(r"//[^\n]*", "", code))]
    assert kinds.count("read") >= 2 and kinds.count("reset") >= 5
    assert _early_resets(code) == []


def test_the_status_word_is_looked_at_together():
    with open(os.path.join(CSRC, "smqa_topk.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    looks = [line for line in code.splitlines() if re.search(r"\*>\(p\.status\)", line)]
    assert looks and all("__syncthreads_or" in line for line in looks)


def test_the_check_itself():
    assert _early_resets("const int m = misc[3], r = 1;\n settle(tk, m, r);") == [2]
    assert _early_resets("const int m = misc[3];\n__syncthreads();\nsettle(tk, m, r);") == []
    assert _early_resets("tk.template reduce<1>(c);\nm = misc[3];\nif (tid == 0) misc[3] = 0;") == [3]
