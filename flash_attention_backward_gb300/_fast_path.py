"""Where the marshalling module of paged.py lies; for build.py and paged.py."""
import os
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))


def fast_path():
    """The module's file.  It is compiled against PyTorch's C++ classes and this interpreter, whose versions
    its name carries: after a change of either the old one is not taken.  None without PyTorch."""
    try:
        import torch
    except ImportError:
        return None
    return os.path.join(HERE, "_fast.torch-%s%s" % (torch.__version__, sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
