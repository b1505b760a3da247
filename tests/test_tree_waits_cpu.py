"""The tree kernels' way out when a bounded wait gives up, read in their sources (it
cannot be provoked on a GPU without a kernel that is broken on purpose): a warp that
shares a named barrier with others leaves by the group's vote only."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_hybrid_attention_gb300", "csrc")
FILES = ["attn_tree_local.cu", "attn_tree_local_rows.cu", "attn_tree_global.cu", "attn_tree_global_rows.cu"]
BARRIER = re.compile(r"softmax_bar\(|bar\.sync|group_all\(")
VOTE = re.compile(r"group_all\(|softmax_bar\(\w*\);\s*const int2 flag = [^;]*;\s*if \(flag\.y\) break;")
END = re.compile(r"kEnd\) \{\s*softmax_bar\(\);[^\n]*\s*break;")


def roles(name):
    """The kernel's warp roles: the text between the ruled headings, helpers left out."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    parts = re.split(r"// -{5,} ?([A-Za-z][^\n]*)\n", text[text.index("__global__"):])
    return dict(zip(parts[1::2], parts[2::2]))


def block(text, start):
    """The braces' block that begins at or after `start`."""
    at, depth = text.index("{", start), 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]


@pytest.mark.parametrize("name", FILES)
def test_groups_leave_together(name):
    groups(name, r"for \(int u = tree_unit", 0 if name == "attn_tree_global_rows.cu" else 1)


def test_decode_group_leaves_together():
    groups("attn_global.cu", r"for \(uint32_t n = 0;; ", 1)


def groups(name, loop, expected):
    found = 0
    for role, text in roles(name).items():
        text = text.split("\n  tc::fence_before();\n  __syncthreads();")[0]
        if not BARRIER.search(text):
            continue
        found += 1
        loops = [block(text, m.start()) for m in re.finditer(loop, text)]
        body = loops[-1]
        assert "group_all(" in body, role
        # no wait that gives up leaves the loop by itself
        assert not re.search(r"!\s*(warp|mbar)_wait\([^;]*\)\s*\)?\s*(\{[^}]*)?break", body), role
        for m in re.finditer(r"if \(([^\n]*)\) break;", body):
            assert m.group(1).strip() in ("!all", "!group_all(1, ok)", "flag.y"), (role, m.group(0))
        if "kEnd" in body:  # the end is met by a vote too
            assert block(body, body.index("d.flags & kEnd")).strip("{ \n").startswith("softmax_bar(")
        # the first barrier behind every wait is a vote: group_all, or a flag set before a barrier and read behind it
        for m in re.finditer(r"(warp|mbar)_wait\(", body):
            after = BARRIER.search(body, m.end())
            assert after is None or VOTE.search(body, after.start()).start() == after.start() or \
                END.search(body, after.start() - 30), (role, body[m.start():m.start() + 60])
    assert found == expected


@pytest.mark.parametrize("name", FILES)
def test_roles_wait_for_what_they_issued(name):
    """Copies and products that are in flight when a role ends are waited for, before the CTA's memory goes."""
    found = {}
    for role, text in roles(name).items():
        loops = [(m.start(), block(text, m.start())) for m in re.finditer(r"for \(int u = tree_unit", text)]
        for start, body in loops:
            behind = text[text.index(body, start) + len(body):].lstrip()
            if re.search(r"tma_rows\(|bulk_g2s\(", body):
                found["copies"] = behind.startswith(("drain<kStages>(", "drain<NB>("))
            elif "commit_warp(" in body:
                found[role.split()[0]] = behind.startswith("drain<")
    assert found == {"copies": True, "Q.K^T": True, "P.V": True}, found
