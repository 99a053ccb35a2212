// Rows of dropout's blocks, on the host: for each "b cols8" of the input, the row.
#include <stdio.h>

#include "slide_rows.h"

int main(void)
{
    long long b, cols8;
    while (scanf("%lld %lld", &b, &cols8) == 2)
        printf("%lld\n", (long long)slide::row_of_block(b, cols8));
    return 0;
}
