"""A replay on the CPU of the MXFP4 ping-pong loop as csrc/gemm_mxfp4.hip has it: the two groups' tick sequences,
branch-free steady state included, are read out of the source, statement by statement, and run against a model of the
memory operations.  Per wave, operations complete in issue order; a wait for at most n outstanding ones completes all
but the last n; a tick's barrier publishes what its waits completed.  Checked for every number of K-steps: what a tick
reads was published before it and is not overwritten; a stage is loaded only after the last read of what it held; every
half K-step is multiplied once, in order; both groups meet at the same number of barriers.  Changed waits, stages and
K-steps, planted in the text, are caught."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routing_grouped_gemm_amd", "csrc",
                      "gemm_mxfp4.hip")


class Bad(Exception):
    pass


def source():
    """The two branches of mainloop4_pp behind its read_all, comments and blanks left out."""
    with open(SOURCE) as f:
        text = f.read()
    body = text[text.index("mainloop4_pp("):]
    body = body[:body.index("\n}\n")]
    main = body[body.index("    if (g == 0) {\n        read_all();"):]
    return body, re.sub(r"//[^\n]*", "", main)


def closing(text, at):
    """Index behind the brace that closes the one at text[at]."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if not depth:
            return i + 1
    raise AssertionError("unbalanced")


def statements(text):
    """A block as a list: simple statements as text, ('for' | 'if', head, block) and ('def', name, block)."""
    out, i = [], 0
    while True:
        while i < len(text) and text[i].isspace():
            i += 1
        if i >= len(text):
            return out
        m = re.compile(r"(for|if) \((.*?)\) \{|auto (generic) = \[&\]\(int end\) __attribute__\(\(always_inline\)\) \{").match(text, i)
        if m:
            end = closing(text, m.end() - 1)
            kind, head = (("def", m[3]) if m[3] else (m[1], m[2]))
            out.append((kind, head, statements(text[m.end():end - 1])))
            i = end + (1 if text[end:end + 1] == ";" else 0)
            continue
        depth, j = 0, i                                   # to the statement's end, past the braces of lambdas
        while depth or text[j] != ";":
            depth += (text[j] in "({[") - (text[j] in ")}]")
            j += 1
        out.append(re.sub(r"\s+", " ", text[i:j]))
        i = j + 1


def split_branches(main):
    a = main.index("{")
    b = closing(main, a)
    rest = main[b:]
    assert rest.lstrip().startswith("else {")
    c = rest.index("{")
    return statements(main[a + 1:b - 1]), statements(rest[c + 1:closing(rest, c) - 1])


def expr(text, env):
    """An index expression of the source."""
    text = text.replace("&&", "and").replace("/", "//")
    assert re.fullmatch(r"[\w\s+\-*<>=!%()]*(and[\w\s+\-*<>=!%()]*)*", text), text
    return eval(text, {"__builtins__": {}}, env)


class Group:
    """One group's program as a list of ticks, each a list of events that its end's barrier closes."""

    def __init__(self, g, nk, program):
        self.g, self.nk, self.ticks, self.now = g, nk, [], []
        self.env = dict(nk=nk, H=2 * nk, STAGE=1)
        self.generic = None
        self.run(program)
        assert not self.now

    def barrier(self):
        self.ticks.append(self.now)
        self.now = []

    # the source's helpers, whose conditions tests/test_mxfp4_schedule_host.py replays by themselves
    def loads(self, t):
        nk = self.nk
        if self.g == 0:
            j = (t + 7) >> 2 if t & 3 == 1 else (t + 5) >> 2
            ops = ("sc", "ha") if t & 3 == 1 else ("hb",)
        else:
            j = (t + 6) >> 2 if t & 3 == 2 else (t + 4) >> 2
            ops = ("sc", "hb") if t & 3 == 2 else ("ha",)
        if 2 <= j < nk:
            for op in ops:
                if op == "sc":
                    if j % 2 == 0:
                        self.now.append(("sc", j >> 1))
                else:
                    self.now.append((op, j & 1, j))

    def waits(self, t):
        nk = self.nk
        if t & 3 == 1:
            j = (t + 3) >> 2
            jn = j + 1 if self.g == 0 else j
            self.now.append(("wait", 0 if jn < 2 or jn >= nk else 5 if self.g == 0 and jn % 2 == 0 else 4))
        elif t & 3 == 2 and self.g == 1:
            jn = ((t + 2) >> 2) + 1
            self.now.append(("wait", 0 if jn < 2 or jn >= nk else 5 if jn % 2 == 0 else 4))

    def run(self, block):
        env = self.env
        for st in block:
            if isinstance(st, tuple):
                kind, head, inner = st
                if kind == "def":
                    self.generic = inner
                elif kind == "if":
                    if expr(head, env):
                        self.run(inner)
                else:
                    init, cond, step = head.split(";")
                    if init.strip():
                        name, value = re.fullmatch(r"int (\w+) = (.+)", init.strip()).groups()
                        env[name] = expr(value, env)
                    while expr(cond, env):
                        self.run(inner)
                        for part in step.split(","):
                            m = re.fullmatch(r"\+\+(\w+)|(\w+) \+= (\d+)", part.strip())
                            env[m[1] or m[2]] += int(m[3] or 1)
                continue
            self.simple(st)

    def simple(self, st):
        env, ev = self.env, self.now
        if st == "read_all()":
            ev.append(("read", 0))
        elif st == "int u = 0":
            env["u"] = 0
        elif re.fullmatch(r"shift\(w[qr]\)", st):
            pass
        elif st == "barrier()":
            self.barrier()
        elif m := re.fullmatch(r"wait_vmcnt<(\d)>\(\)", st):
            ev.append(("wait", int(m[1])))
        elif m := re.fullmatch(r"sc\.issue\((.+)\)", st):
            ev.append(("sc", expr(m[1], env)))
        elif m := re.fullmatch(r"(ha|hb)\.issue\((.+), (.+)\)", st):
            ev.append((m[1], expr(m[2], env), expr(m[3], env)))
        elif m := re.fullmatch(r"loads\((.+)\)", st):
            self.loads(expr(m[1], env))
        elif m := re.fullmatch(r"end_tick\((.+)\)", st):
            self.waits(expr(m[1], env))
            self.barrier()
        elif m := re.fullmatch(r"generic\((.+)\)", st):
            env["end"] = expr(m[1], env)
            self.run(self.generic)
        elif m := re.fullmatch(r"last\((.+)\)", st):
            ev.append(("multiply", None))
            self.waits(expr(m[1], env))
            self.barrier()
        elif m := re.fullmatch(r"compute\(rd, (odd|even), (.+?), sp, s[qr], s[qr], w[qr], w[qr], (.+)\)", st):
            hs = expr(m[2], env)
            assert hs % 2 == (m[1] == "odd")
            ev += [("multiply", hs - 1), ("read", hs)]
            if w := re.fullmatch(r"\[&\] \{ waits\((.+)\); \}", m[3]):
                self.waits(expr(w[1], env))
            else:
                assert m[3] in ("none", "wait4"), m[3]
                if m[3] == "wait4":
                    ev.append(("wait", 4))
            self.barrier()
        else:
            raise AssertionError("a statement that the replay does not know: " + st)


def replay(nk, branches):
    groups = [Group(g, nk, branches[g]) for g in (0, 1)]
    H = 2 * nk
    if len(groups[0].ticks) != len(groups[1].ticks):
        raise Bad("the groups meet at different numbers of barriers")
    queue, done, held, last_read, mult = {0: [], 1: []}, {}, {}, {}, {0: [], 1: []}
    names = {(0, "ha"): "a0", (1, "ha"): "a1", (0, "hb"): "b1", (1, "hb"): "b0", (0, "sc"): "As", (1, "sc"): "Bs"}

    def issue(g, t, op, stage, j, n):
        name = names[g, op]
        if j >= (nk if op != "sc" else (nk + 1) // 2):
            raise Bad(f"{name} {j} lies past the operand")
        if (name, stage) in held and last_read.get(held[name, stage], -99) >= t:
            raise Bad(f"{name} {j} overwrites {held[name, stage]} at tick {t}")
        held[name, stage] = (name, j)
        queue[g] += [(name, j)] * n

    def wait(g, t, n):
        q = queue[g]
        keep = q[len(q) - n:] if n else []
        for item in q[:len(q) - n] if n else q:
            if item not in keep:
                done.setdefault(item, t)
        queue[g] = keep

    for g in (0, 1):                                      # ahead of the loop
        issue(g, -9, "sc", 0, 0, 1)
        for j in range(min(nk, 2)):
            issue(g, -9, "ha", j, j, 4)
            issue(g, -9, "hb", j, j, 4)
        wait(g, -1, 8 if nk > 1 else 0)
    for t in range(len(groups[0].ticks)):
        for g in (0, 1):
            for e in groups[g].ticks[t]:
                if e[0] == "read":
                    j, c = e[1] >> 1, e[1] >> 2
                    for item, stage in (((f"a{g}", j), j & 1), (("b0", j), j & 1), (("b1", j), j & 1), (("As", c), c & 1),
                                        (("Bs", c), c & 1)):
                        if done.get(item, 1 << 30) >= t or held.get((item[0], stage)) != item:
                            raise Bad(f"group {g} reads {item} at tick {t}")
                        last_read[item] = t
                elif e[0] == "multiply":
                    mult[g].append(e[1])
        # a load may land at once, so it counts against the other group's reads of the same tick too
        for g in (0, 1):
            for e in groups[g].ticks[t]:
                if e[0] == "sc":
                    issue(g, t, "sc", e[1] & 1, e[1], 1)
                elif e[0] in ("ha", "hb"):
                    issue(g, t, e[0], e[1], e[2], 4)
                elif e[0] == "wait":
                    wait(g, t, e[1])
    for g in (0, 1):
        if mult[g] != list(range(H - 1)) + [None]:
            raise Bad(f"group {g} multiplies {mult[g]}")


@pytest.mark.parametrize("nk", list(range(1, 45)))
def test_loop_of_the_source(nk):
    replay(nk, split_branches(source()[1]))


def test_helpers_are_those_of_the_source():
    """The conditions that Group.loads and Group.waits repeat, and the order of operations ahead of the loop."""
    body, _ = source()
    flat = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", body))
    for text in (
        "if ((t & 3) == 1) { j = (t + 7) >> 2; if (j >= 2 && j < nk) { if ((j & 1) == 0) sc.issue(j >> 1); "
        "ha.issue((uint32_t)(j & 1) * STAGE, j); } } else { j = (t + 5) >> 2; "
        "if (j >= 2 && j < nk) hb.issue((uint32_t)(j & 1) * STAGE, j); }",
        "if ((t & 3) == 2) { j = (t + 6) >> 2; if (j >= 2 && j < nk) { if ((j & 1) == 0) sc.issue(j >> 1); "
        "hb.issue((uint32_t)(j & 1) * STAGE, j); } } else { j = (t + 4) >> 2; "
        "if (j >= 2 && j < nk) ha.issue((uint32_t)(j & 1) * STAGE, j); }",
        "if ((t & 3) == 1) { const int j = (t + 3) >> 2; const int jn = g == 0 ? j + 1 : j; "
        "if (jn < 2 || jn >= nk) wait_vmcnt<0>(); else if (g == 0 && (jn & 1) == 0) wait_vmcnt<5>(); "
        "else wait_vmcnt<4>(); } else if ((t & 3) == 2 && g == 1) { const int jn = ((t + 2) >> 2) + 1; "
        "if (jn < 2 || jn >= nk) wait_vmcnt<0>(); else if ((jn & 1) == 0) wait_vmcnt<5>(); else wait_vmcnt<4>(); }",
        "auto wait4 = []() __attribute__((always_inline)) { wait_vmcnt<4>(); };",
        "sc.issue(0); ha.issue(0, 0); hb.issue(0, 0); if (nk > 1) { ha.issue(STAGE, 1); hb.issue(STAGE, 1); "
        "wait_vmcnt<8>(); } else { wait_vmcnt<0>(); } __syncthreads();",
    ):
        assert text in flat, text


@pytest.mark.parametrize("old,new", [
    ("wait_vmcnt<5>();", "wait_vmcnt<9>();"), ("wait_vmcnt<4>();", "wait_vmcnt<8>();"), ("wq, wr, wait4)", "wq, wr, none)"),
    ("ha.issue(0, 2 * c + 2);", "ha.issue(STAGE, 2 * c + 2);"), ("hb.issue(STAGE, 2 * c + 3);", "hb.issue(STAGE, 2 * c + 4);"),
    ("sc.issue(c + 1);", "sc.issue(c + 2);"), ("int c = 1;", "int c = 0;"), ("generic(5);", "generic(7);"),
    ("++c, u += 4", "++c, u += 2"),
])
def test_planted_mistakes_are_caught(old, new):
    _, main = source()
    assert main.count(old) >= 1
    at = [m.start() for m in re.finditer(re.escape(old), main)]
    for i in at:                                          # each place by itself
        wrong = split_branches(main[:i] + new + main[i + len(old):])
        with pytest.raises(Bad):
            for nk in range(1, 30):
                replay(nk, wrong)
