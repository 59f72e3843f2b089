"""What the update's kernels do once a bounded wait has run out, read from their source (the
bounded-wait tests issue no MMAs, so that none is in flight when theirs do)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "activated_mlp_gemms_gb300", "csrc")


def kernels(name):
    """(name, body) of a file's kernels, without comments."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    found = []
    for start in re.finditer(r"__global__[^;{]*?(k_\w+)\(", src):
        at = src.index("{", start.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
            if depth == 0:
                break
        found.append((start.group(1), src[at:end]))
    return found


@pytest.mark.parametrize("file,names", [("k_ortho.cu", {"k_ortho_gemm", "k_ortho_split"}),
                                        ("k_ortho_small.cu", {"k_ortho_small"})])
def test_mmas_end_before_tensor_memory_is_freed(file, names):
    # a kernel that gives up commits what it has issued to a barrier of its own and waits for it
    # (with a limit that no other wait's failure cuts short) before it frees tensor memory
    seen = set()
    for name, body in kernels(file):
        if "tmem_dealloc" not in body:
            continue
        seen.add(name)
        free = body.index("tmem_dealloc")
        commit = re.search(r"tc_commit\((?:bar_s\(DRAIN\)|drain)\)", body[:free])
        assert commit, name
        wait = re.search(r"mbar_wait(?:<\w+>)?\((?:bar_s\(DRAIN\)|drain), 0, \d+ull, &never\)",
                         body[commit.end():free])
        assert wait, name
    assert seen == names


def test_the_small_kernel_issues_nothing_after_a_failed_wait():
    # its steps go on (the cluster's barriers are matched), its one barrier's phases do not: a
    # round that ends late must not be taken for a later one
    (_, body), = kernels("k_ortho_small.cu")
    issue = body.index("issue();")
    guard = body.rindex("if (", 0, issue)
    assert "!*abort_flag" in body[guard:issue]
    assert re.search(r"__syncthreads\(\);\s*if \([^)]*$", body[:body.index("!*abort_flag")])
    assert re.search(r"if \(ok && !mbar_wait\(bar, phase,", body)


def test_the_skinny_linear_kernel_waits_for_what_it_issued():
    # its MMA warp commits what it has issued, also when it gives up; a failure elsewhere cuts the
    # other warps' wait for that short, so that they wait once more, whatever has failed
    body = next(b for _, b in kernels("k_linear_skinny.cu") if "tmem_dealloc" in b)
    first = body.index("const bool summed = mbar_wait(done, 0,")
    again = re.search(r"if \(!summed\) \{[^}]*mbar_wait\(done, 0, \d+ull, &never\);", body[first:])
    assert again and first + again.end() < body.index("tmem_ld16")
