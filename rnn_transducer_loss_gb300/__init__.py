"""rnn_transducer_loss_gb300: fused RNN-T (transducer) loss forward+backward for GB300,
and the label side of a transducer around it: label embedding and its gradient
for training, beam selection and reordering of states for decoding.

The compute path is a C-ABI shared library (``librnnt_gb300.so``, declared in
``include/rnnt_gb300.h``) of hand-written CUDA kernels for sm_103a.  This
package only marshals arguments to it: ``rnnt_loss`` allocates outputs and the
workspace with PyTorch and passes raw device pointers and the current stream.
The library is loaded on first use and a missing library raises; there is no
other implementation to fall back to.
"""
_FROM = {"rnnt_loss": "functional", "RNNTLoss": "functional",
         "rnnt_embed": "embedding", "rnnt_embed_grad": "embedding", "RNNTEmbedding": "embedding",
         "rnnt_beam_select": "beam", "rnnt_beam_reorder": "beam"}
__all__ = list(_FROM)


def __getattr__(name):
    if name in _FROM:
        from importlib import import_module
        value = getattr(import_module("." + _FROM[name], __name__), name)
        globals()[name] = value
        return value
    raise AttributeError(name)
