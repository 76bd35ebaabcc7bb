// Attention of a tree of drafts, many rows: the tensor-memory kernel with a mask a draft.
#define KDA_ATTN_TREE
#include "attn_prefill.cu"
