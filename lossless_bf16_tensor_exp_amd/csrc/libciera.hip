// libciera.hip -- the library's one translation unit: the lossless codec, then
// the microscaled matrices, which share its status words and launches.
#include "ciera.hip"
#include "mx.hip"
