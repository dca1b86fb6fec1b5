"""The text of a CUDA kernel as a tree of blocks, for tests of orders that a run
cannot show (a missing wait that happens to be harmless on an idle GPU)."""
from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rope_rope3d_apply_gb300", "csrc")


class Block:
    """A braced block: `head` is what stands before its brace, `parts` its text
    pieces (str) and inner blocks in order."""

    def __init__(self, head):
        self.head, self.parts = head, []


def kernel(file, name):
    """The body of __global__ function `name` (comments taken out)."""
    with open(os.path.join(CSRC, file)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = re.search(r"__global__[^;{}]*\b" + name + r"\s*\([^{]*\{", text).end()
    root = Block(name)
    stack, start = [root], at
    for i in range(at, len(text)):
        c = text[i]
        if c == "{":
            piece = text[start:i]
            depth, j = 0, len(piece)   # back to the last ; or } outside parentheses
            while j > 0 and not (depth == 0 and piece[j - 1] in ";}"):
                depth += {")": 1, "(": -1}.get(piece[j - 1], 0)
                j -= 1
            head = piece[j:].strip()
            stack[-1].parts.append(piece)
            inner = Block(head)
            stack[-1].parts.append(inner)
            stack.append(inner)
            start = i + 1
        elif c == "}":
            stack[-1].parts.append(text[start:i])
            start = i + 1
            stack.pop()
            if not stack:
                return root
    raise AssertionError(f"{name}: unbalanced braces")


def flat(block) -> str:
    """The block's whole text again, braces included."""
    return "".join(p if isinstance(p, str) else "{" + flat(p) + "}" for p in block.parts)


def before_each(block, wanted, needed, seen=False, missing=None):
    """Which uses of `wanted` (a call's name) no use of `needed` stands before on
    their way: (whether `needed` has happened at the block's end, the texts before
    those uses). Both branches of an if / else count together."""
    missing = [] if missing is None else missing
    call = re.compile(r"\b(?:" + wanted + r"|" + needed + r")\s*\(")
    branches = []   # of the if / else chain being read: needed has happened at their ends
    for i, part in enumerate(block.parts):
        if isinstance(part, str):
            is_else = part.strip().startswith("else")
            if branches and not is_else:
                # a chain without a last else may be passed by
                seen = seen or (branches[-1][1] and all(b for b, _ in branches))
                branches = []
            for m in call.finditer(part):
                if m.group().startswith(needed):
                    seen = True
                elif not seen:
                    missing.append((block.head + ": " + part[max(0, m.start() - 60):m.end()]).strip())
            continue
        conditional = re.search(r"\b(if|else|for|while)\b", part.head) is not None
        chained = re.search(r"\b(if|else)\b", part.head) is not None
        end, _ = before_each(part, wanted, needed, seen, missing)
        if chained:
            branches.append((end, re.search(r"\bif\b", part.head) is None))
        elif not conditional:
            seen = end
    if branches:
        seen = seen or (branches[-1][1] and all(b for b, _ in branches))
    return seen, missing
