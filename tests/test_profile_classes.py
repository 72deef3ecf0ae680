"""The profiling hook's kernel classes: the header and the binding name the same ones."""
import os
import re

from text_embedding_encoder_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_binding_names_the_header_s_classes():
    text = open(os.path.join(ROOT, "include", "tee.h")).read()
    classes = {m[0].lower(): int(m[1]) for m in re.findall(r"^#define TEE_K_(\w+)\s+(\d+)", text, flags=re.M)}
    assert classes.pop("count") == len(binding.KERNEL_CLASSES)
    assert classes == {name: i for i, name in enumerate(binding.KERNEL_CLASSES)}
