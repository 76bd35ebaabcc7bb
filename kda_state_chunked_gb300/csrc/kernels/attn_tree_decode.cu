// Attention of a tree of drafts, few rows: the register kernel with a mask a draft.
#define KDA_ATTN_TREE
#include "attn_decode.cu"
