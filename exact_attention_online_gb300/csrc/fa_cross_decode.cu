// Decoding attention over contiguous K and V: the kernels of the paged cache for a pool of one
// page a sequence, without a table.
#define FA_CONTIGUOUS 1
#include "fa_paged.cu"
