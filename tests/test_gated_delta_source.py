"""Rules that the chunked kernel's source has to keep, checked by reading it.

A wait on an mbarrier does not by itself order a thread's tensor-memory accesses
after those that the barrier stands for: tcgen05.fence::after_thread_sync has to
come between.  Where one is missing the results are right as long as the timing
is, so no run shows it.
"""
import os
import re

import selective_state_space_conv1d_gb300 as m

_CSRC = os.path.join(os.path.dirname(m.__file__), "csrc")


def _roles():
    """The chunk kernel's text by role: epilogues, prepare, gates, MMAs, load."""
    with open(os.path.join(_CSRC, "gated_delta_chunk.cu")) as f:
        text = re.sub(r"//(?! -----).*", "", f.read())  # without comments, but for the roles' headings
    parts = re.split(r"// -{10,} (\w+) -{4}", text)
    return dict(zip(parts[1::2], parts[2::2]))


def _unfenced(text, wait, access):
    """Accesses whose last wait before them has no fence between."""
    bad, pending = [], None
    for e in re.finditer(rf"(?P<wait>{wait})|(?P<fence>\btcgen05_fence_after\(\))|(?P<access>{access})", text):
        if e["wait"]:
            pending = e["wait"]
        elif e["fence"]:
            pending = None
        elif pending:
            bad.append((pending, e["access"]))
    return bad


def test_products_come_after_a_fence():
    text = _roles()["MMAs"]
    assert text.count("wait_counted(") >= 8
    assert _unfenced(text, r"\bwait_counted\([a-z_0-9]+", r"\b(?:issue_d[01]|mma_ss|mma_ts)\(") == []


def test_tensor_memory_is_touched_after_a_fence():
    """Behind the barriers that products commit to, in the warps that load and store tensor memory."""
    for role in ("epilogues", "prepare"):
        text = _roles()[role]
        assert re.search(r"\bwait\((?:[xuso]|d0)_full", text)
        assert _unfenced(text, r"\bwait\((?:[xuso]|d0)_full", r"\btmem_(?:ld|st)\d+\(") == []


def _lambda(text, name):
    """The text of `auto name = [&](..) {..};`."""
    start = text.index(f"auto {name} = [&](")
    depth = 0
    for i in range(text.index("{", start), len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]


def test_no_barrier_hangs_on_what_the_gates_say():
    """Once a wait has run out, the gates of a chunk may be unwritten and differ between warps' reads."""
    text = _roles()["epilogues"]
    for name in ("enter", "leave"):  # both run, or not, by the gates
        assert "named_barrier(" not in _lambda(text, name) and "__syncthreads(" not in _lambda(text, name)


def test_no_address_is_made_of_an_aborted_chunk_s_gates():
    """Each use of the gates for a global address looks at the abort flag between reading them and the access."""
    text = _roles()["epilogues"]
    for name in ("enter", "leave"):
        body = _lambda(text, name)
        read, access = body.split("if (!live()) return;")
        assert re.search(r"\bk\.bh\b", read)
        # k.phi of enter chooses no address
        assert not re.search(r"\bk\.(?!phi\b)\w+", access) and not re.search(r"(?:load|store)_state\(", read)
    output, values = _lambda(text, "output"), text[text.index("epilogue 1" if "epilogue 1" in text else "float r[kTok];"):]
    assert re.search(r"y_rows = [^;]*gt\.tokens[^;]*;\s*if \(!live\(\)\) y_rows = 0;", output)
    assert re.search(r"int rows = [^;]*gt\.tokens[^;]*;[^;]*;\s*if \(!live\(\)\) rows = 0;", values)


def test_nothing_is_in_flight_when_a_cta_ends():
    """A wait that ran out leaves copies and products in flight: they are waited for before the memory is given back."""
    mma, load = _roles()["MMAs"], _roles()["load"]
    end = mma[mma.rindex("issue_d0("):]
    assert re.search(r"\bcommit\(drained\);\s*landed\(drained, 0\);", end) and "wait_counted(" not in end
    copies = [c.start() for c in re.finditer(r"\bmbar_arrive_expect_tx\(", load)]
    assert len(copies) == 2
    for at, name in zip(copies, ("kq", "v")):  # none is started after the flag is up
        assert re.search(rf"if \(lt == 0 && !\*abort_flag\) \{{\s*{name}_started = c \+ 1;\s*$", load[:at])
    rest = load[load.index("if (MAPS && lt == 0 && *abort_flag)"):]
    assert re.search(r"landed\(kq_full", rest) and re.search(r"landed\(v_full", rest)
    # before the barrier of the values is used for anything else
    assert rest.index("landed(v_full") < rest.index("mbar_arrive(v_full)")
