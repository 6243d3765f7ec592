// libciera.hip -- the library's one translation unit: the lossless codec, the
// microscaled matrices, which share its status words and launches, and what
// stands around their products in a layer.
#include "ciera.hip"
#include "mx.hip"
#include "norm.hip"
#include "experts.hip"
#include "low_rank.hip"
