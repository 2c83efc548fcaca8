"""A tree of drafted tokens over the paged int8 cache: the newest rows of a sequence are the tree's nodes, row j
continuing row parent[j] (an earlier one, or -1: the cached context).  One step:

    mask, pos = tw.draft_tree_mask(batch, parent, words)             # once for all layers
    q = tw.i8_kv_append(cache, batch, f, k, v, q=q, pos=pos)         # a layer
    o = tw.i8_kv_attend_tree(cache, batch, q, mask)
    ...                                                              # head: target = argmax of every row
    path, count, following = tw.draft_tree_accept(batch, parent, token, target)
    lens = tw.i8_kv_keep(cache, batch, tokens, path)                 # a layer
"""
from __future__ import annotations

import ternary_weight_decode_amd as _tw

# These calls take as long as their launches: what they need is looked up once.
_torch = _tw._setup()
_lib = _tw.lib()
_i64c = _tw._i64
_i32, _i64, _bf16 = _torch.int32, _torch.int64, _torch.bfloat16
TREE_ROWS = 512
TREE_WORDS = TREE_ROWS // 64


def _int32(t, name, shape, device):
    _tw._vec(t, name, _i32, shape, device)


def _parents(parent, device):
    """Rows of the batch, one parent each."""
    if not isinstance(parent, _torch.Tensor) or parent.dim() != 1:
        _int32(parent, "parent", (None,), device)
    n = parent.shape[0]
    _int32(parent, "parent", (n,), device)
    return n


def draft_tree_mask(batch, parent, words: int = 1, mask=None, pos=None, stream=None):
    """Who descends from whom: parent int32 [T] -> (mask int64 [T, words], 64 rows of the tree to a word;
    pos int32 [T], the positions for the rotation).  words: enough for the largest tree, at most 8."""
    device = batch.device
    tokens = _parents(parent, device)
    if not 1 <= words <= TREE_WORDS:
        raise RuntimeError(f"words is {words}, expected 1 to {TREE_WORDS}")
    if mask is None:
        mask = _tw._empty(_i64, device, stream, tokens, words)
    else:
        _tw._vec(mask, "mask", _i64, (tokens, words), device)
    if pos is None:
        pos = _tw._empty(_i32, device, stream, tokens)
    else:
        _int32(pos, "pos", (tokens,), device)
    _tw._launch(_lib.draft_tree_mask, device, stream, batch.ref, tokens, parent.data_ptr(), words, mask.data_ptr(),
                pos.data_ptr())
    return mask, pos


def i8_kv_attend_tree_workspace_bytes(tokens: int, hq: int, heads: int, d: int, nseq: int, max_len: int) -> int:
    """Bytes that i8_kv_attend_tree needs for exactly these sizes and this max_len; smaller ones may need more."""
    return int(_lib.i8_kv_attend_tree_workspace_bytes(tokens, hq, heads, d, nseq, max_len))


def i8_kv_attend_tree_workspace_limit(tokens: int, hq: int, heads: int, d: int, nseq: int) -> int:
    """Bytes that serve every call of up to `tokens` rows and nseq sequences, whatever its max_len."""
    return int(_lib.i8_kv_attend_tree_workspace_limit(tokens, hq, heads, d, nseq))


def i8_kv_attend_tree_workspace(cache, batch, tokens: int, hq: int, max_len=None):
    """A workspace for i8_kv_attend_tree of up to `tokens` rows of hq heads and the batch's number of sequences: as
    large as any of these calls needs, whatever its max_len (None where there is nothing to do)."""
    nbytes = i8_kv_attend_tree_workspace_limit(tokens, hq, cache.heads, cache.d, batch.nseq)
    if nbytes < 0 or (max_len is not None and not 0 < max_len < 2 ** 31):
        _tw._check("i8_kv_attend_tree_workspace", 2)
    return _torch.empty(nbytes, dtype=_torch.uint8, device=cache.device) if nbytes else None


def i8_kv_attend_tree_config(tokens: int, hq: int, heads: int, d: int, nseq: int, width: int, max_len=None):
    """The kernel that i8_kv_attend_tree takes for `tokens` rows of hq heads (host-side, no device needed; width:
    of the table, max_len by default what that holds): a dict, empty where there is nothing to do."""
    out = (_i64c * 3)()
    rc = _lib.i8_kv_attend_tree_config(tokens, hq, heads, d, nseq, width,
                                       max(1, width * _tw.KV_BLOCK) if max_len is None else max_len, out)
    if rc < 0:
        _tw._check("i8_kv_attend_tree_config", -rc)
    return dict(zip(("cols", "groups", "grid"), map(int, out))) if rc else {}


def i8_kv_attend_tree(cache, batch, q, mask, scale=None, max_len=None, out=None, workspace=None, stream=None):
    """Attention of q bf16 [T, Hq, D] over the batch's cached tokens -> bf16 [T, Hq, D]: a row sees what stands in
    front of its tree, and of the tree the rows up to its own whose bits its mask has (int64 [T, words]).
    scale: D ** -0.5 by default.  max_len: the longest length that batch.lens will hold, a hint (default: what
    the table can hold)."""
    device, d = _tw._kv_device(cache, batch), cache.d
    tokens, hq, stride = _tw._rows(q, "q", _bf16, device, None, d, None)
    if not isinstance(mask, _torch.Tensor) or mask.dim() != 2:
        _tw._vec(mask, "mask", _i64, (tokens, None), device)
    words = mask.shape[1]
    _tw._vec(mask, "mask", _i64, (tokens, words), device)
    if max_len is None:
        max_len = batch.width * _tw.KV_BLOCK or 1
    if out is None:
        out = _tw._empty(_bf16, device, stream, tokens, hq, d)
    else:
        _tw._vec(out, "out", _bf16, (tokens, hq, d), device)
    need = _lib.i8_kv_attend_tree_workspace_bytes(tokens, hq, cache.heads, d, batch.nseq, max_len)
    if workspace is None:
        if need > 0:
            workspace = _tw._new(need, _torch.uint8, device, stream, returned=False)
    elif workspace.get_device() != device or not workspace.is_contiguous() or workspace.nbytes < need:
        raise RuntimeError(f"workspace must be a contiguous tensor of at least {need} bytes on device {device}")
    _tw._launch(_lib.i8_kv_attend_tree, device, stream, cache.ref, batch.ref, tokens, q.data_ptr(), hq, stride,
                d ** -0.5 if scale is None else scale, mask.data_ptr(), words, max_len, out.data_ptr(),
                _tw._addr(workspace))
    return out


def draft_tree_accept(batch, parent, token, target, width: int = 64, path=None, count=None, following=None,
                      stream=None):
    """The branch that the target's own tokens take: token int32 [T], what a row carries; target int32 [T], what the
    target answers there -> (path int32 [nseq, width], rows of each tree and then -1; count int32 [nseq];
    following int32 [nseq], the target's token behind the last)."""
    device, nseq = batch.device, batch.nseq
    tokens = _parents(parent, device)
    _int32(token, "token", (tokens,), device)
    _int32(target, "target", (tokens,), device)
    if path is None:
        path = _tw._empty(_i32, device, stream, nseq, width)
    else:
        _int32(path, "path", (nseq, width), device)
    if count is None:
        count = _tw._empty(_i32, device, stream, nseq)
    else:
        _int32(count, "count", (nseq,), device)
    if following is None:
        following = _tw._empty(_i32, device, stream, nseq)
    else:
        _int32(following, "following", (nseq,), device)
    _tw._launch(_lib.draft_tree_accept, device, stream, batch.ref, tokens, parent.data_ptr(), token.data_ptr(),
                target.data_ptr(), width, path.data_ptr(), count.data_ptr(), following.data_ptr())
    return path, count, following


def i8_kv_keep(cache, batch, tokens: int, path, lens_out=None, stream=None):
    """Of the batch's `tokens` newest rows only those of path int32 [nseq, width] stay in the cache, moved up to
    where their tree began -> int32 [nseq], the lengths to go on with."""
    device = _tw._kv_device(cache, batch)
    if not isinstance(path, _torch.Tensor) or path.dim() != 2:
        _int32(path, "path", (batch.nseq, None), device)
    width = path.shape[1]
    _int32(path, "path", (batch.nseq, width), device)
    if lens_out is None:
        lens_out = _tw._empty(_i32, device, stream, batch.nseq)
    else:
        _int32(lens_out, "lens_out", (batch.nseq,), device)
        if abs(lens_out.data_ptr() - batch.lens.data_ptr()) < 4 * batch.nseq:
            raise RuntimeError("lens_out must not be the batch's lens")
    _tw._launch(_lib.i8_kv_keep, device, stream, cache.ref, batch.ref, tokens, path.data_ptr(), width,
                lens_out.data_ptr())
    return lens_out
